// The gated delta rule over a step's rows (gfx950): trees, single rows and
// short chains (long chains: delta_chain.hip).
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
// Value dims are independent of each other: a wave owns 16 of them
// and holds its columns of S0 in registers, in the layout of the products, so
// states, deltas and results pass from one product into the next without
// leaving the registers.
//
// Precision: q and k are bf16 and enter as they are. A state or delta (fp32)
// enters a bf16 product as three bf16 pieces, each the top of what the one
// before left, which hold all its 24 bits; products of two fp32 factors (L and
// D (q . k) with deltas) run on the fp32 matrix core. Sums of g are held in 64 bits.
//
// Bound by the state's bytes where there are many sequences: 24 x 8 rows, 16 key
// and 48 value heads of 128 x 128, 24.5 us for 85 MB (3.5 TB/s), 32 x 1 41 us for 202 MB
// read and written (4.9 TB/s); by latency where there are few: one 32-row tree
// takes 9.0 us, about 1.5 of them until a sequence's rows and slot are there,
// 2 for the loads behind those, 2.5 for tiles and inverses, 1 for the products;
// 2 are not told apart (start and end, outputs, instructions fetched for the first time).
// A workgroup's code runs once, so its instructions are fetched as it goes:
// loops of few instructions beat unrolled ones outside the state's registers.
#include "delta_mfma.h"
#include "delta_rule.h"

namespace w12 {
namespace {

template <int KD, int RT>
struct Shared {
  static constexpr int R = 16 * RT;
  static constexpr int KS = KD + 8;                 // row of q and k: each 4 banks (of 64) further, so 8-byte reads meet none twice
  static constexpr int TS = 24;                     // the same for a key dim's rows
  alignas(16) uint16_t q[R * KS];
  alignas(16) uint16_t k[R * KS];
  // chains (RT 1): k with rows innermost; trees: the rows of an earlier block
  alignas(16) uint16_t t[RT == 1 && KD * TS > R * KS ? KD * TS : R * KS];
  f32x4 low[RT * RT][64];   // tiles of -L, and
  f32x4 see[RT * RT][64];   // of D (q . k): lane (g, i) holds row i, columns 4 g + r
  f32x4 far_low[RT * RT][64], far_see[RT * RT][64];  // the same against an earlier block of a tree
  f32x4 inv[RT][64];        // (I + L)^-1 of the diagonal tiles
  // by the sequence's row:
  double sum[kStepRows];              // of g from the state (chains: the block) to the row
  unsigned long long in[kStepRows];   // the row's path within its block, itself included
  int16_t leave[kStepRows];           // the row above that, in an earlier block, or below 0
  float beta[kStepRows], grow[kStepRows];  // beta, e^G
  float part[R];                        // chains: e^(G_n - G_j)
  unsigned long long odd[kStepRows / R];  // rows of each block that hold no numbers; of a tree's earlier blocks, those behind such rows too
  unsigned long long odd_q;             // queries of the block that are no numbers
  unsigned long long cross[R];          // the path's rows in an earlier block
  int next[R];                          // where the path leaves that block
  int behind[R];                        // a row on the path in an earlier block holds no number
  int bad;
};

// Rows of keys or queries in the registers of a workgroup, then into LDS, rows past `n` zero. A row with an
// infinity or NaN is marked, and zeros stand in for it: its outputs are set apart from the products.
template <int KD, int R, int kThreads>
struct Staged {
  static constexpr int kChunks = KD / 8, kTurns = (R * kChunks + kThreads - 1) / kThreads;
  uint4 x[kTurns];
  __device__ __forceinline__ void load(const uint16_t* from, int step, int n) {
    const int tid = thread_now();
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
      const int e = tid + i * kThreads;
      x[i] = *reinterpret_cast<const uint4*>(behind(from, 2 * (__umul24(min(e / kChunks, n - 1), step) + (e % kChunks) * 8)));
    }
  }
  __device__ __forceinline__ void store(int n, uint16_t* to, int stride, unsigned long long* odd) {
    const int tid = thread_now();
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
      const int e = tid + i * kThreads, r = e / kChunks;
      if (R * kChunks % kThreads != 0 && e >= R * kChunks) break;
      const bool no = is_odd(odd_sum(x[i]));
      if (no && r < n) atomicOr(odd, 1ull << r);
      if (no || r >= n) x[i] = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(to + r * stride + (e % kChunks) * 8) = x[i];
    }
  }
};

template <int KD, int VD, int RT, int kWaves>
__global__ __launch_bounds__(64 * kWaves, RT == 1 ? 4 : RT == 2 ? 2 : 1) void delta_rule_kernel(DeltaRuleArgs a) {
  constexpr int kThreads = 64 * kWaves;
  using Sh = Shared<KD, RT>;
  constexpr int R = Sh::R, KS = Sh::KS, TS = Sh::TS, KT = KD / 16;
  __shared__ Sh s;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int hv = a.c.value_heads;
  constexpr int slabs = VD / (kWaves * 16);
  const int head = blockIdx.x / slabs, key = head / (hv / a.c.key_heads), seq = blockIdx.y;
  const int vw = (blockIdx.x - head * slabs) * (kWaves * 16) + wave * 16;  // the wave's first value dim
  const RowsView v = rows_view(a.c, a.st, seq);
  if (v.rows == 0) return;
  float* state = a.c.state + state_at(a.c, a.layer, v.slot, head);
  f32x4 S[KT][1];
  // loads come back in order: what is needed before the state is read before it
  const Look seen = look(a, v);
  if (v.rows == 1) {
    load_state<KT, VD, 1>(state, vw, S);
    rows_in_turn<KD, VD, 1>(a, v, seq, head, key, vw, state, seen, S);
    return;
  }
  const bool chain = RT == 1 && !a.st.parent;
  const int blocks = (v.rows + R - 1) / R;
  // a block's keys, queries and values (in the layout of the products)
  Staged<KD, R, kThreads> keys, queries;
  uint32_t values[RT][4];
  const auto fetch = [&](int b) {
    const int row0 = v.row0 + b * R, n = min(R, v.rows - b * R);
    const uint16_t* kv = a.c.kv + kv_at(a.c, a.layer, row0);
    keys.load(kv + key * KD, a.c.kv_width, n);
    queries.load(a.q + ((size_t)row0 * a.c.key_heads + key) * KD, a.c.key_heads * KD, n);
    const int lane = thread_now() & 63, g = lane >> 4, v0 = a.c.key_heads * KD + head * VD + vw + (lane & 15);
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint16_t* p = behind(kv, 2 * (__umul24(min(16 * m + 4 * g + r, n - 1), a.c.kv_width) + v0));
        values[m][r] = *p;
      }
  };
  // parts that one wave plays go round the waves with the workgroup, so that no SIMD has them all
  const int role = (wave + blockIdx.x) & (kWaves - 1);
  float gate0, beta0;  // of the first row whose path this lane follows
  int parent0;
  {
    const int i = min(role * 64 + (thread_now() & 63), v.rows - 1);
    gate0 = a.c.gates[gate_at(a.c, a.layer, v.row0 + i, 0, head)];
    beta0 = a.c.gates[gate_at(a.c, a.layer, v.row0 + i, 1, head)];
    parent0 = a.st.parent ? a.st.parent[v.row0 + i] : i - 1;
  }
  fetch(0);
  load_state<KT, VD, 1>(state, vw, S);
  for (int i = tid; i < kStepRows / R; i += kThreads) s.odd[i] = 0;
  if (tid == 0) s.odd_q = 0, s.bad = 0;
  __syncthreads();
  if (role == kWaves - 1) {
    const int bad = refused(a, v, seq, seen);
    if ((thread_now() & 63) == 0) s.bad = bad;
  }
  // paths within each block, by doubling; a lane is a row, the waves take 64 rows in turn
  for (int i0 = role * 64; i0 < v.rows; i0 += kThreads) {
    const int lane = thread_now() & 63, i = i0 + lane, first = lane & ~(R - 1), row = lane - first;
    float gate = 0, beta = 0;
    int cur = -1, leave = -1;
    if (i < v.rows) {
      const bool again = i0 >= kThreads;
      gate = again ? a.c.gates[gate_at(a.c, a.layer, v.row0 + i, 0, head)] : gate0;
      beta = again ? a.c.gates[gate_at(a.c, a.layer, v.row0 + i, 1, head)] : beta0;
      if (!(gate <= 3.4e38f) || odd32(beta)) {
        atomicOr(&s.odd[i / R], 1ull << row);
        gate = beta = 0;
      }
      int p = chain ? (row > 0 ? i - 1 : -1) : again ? a.st.parent[v.row0 + i] : parent0;
      if (p >= i || p < -1) p = -1;  // no tree: reported, once every row has been looked at
      cur = p - (i - row);
      leave = p;
    }
    double sum = log_decay(gate);
    unsigned long long in = 1ull << row;
#pragma unroll
    for (int step = 1; step < R; step <<= 1) {
      const int from = first + max(cur, 0);
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
    if (i < kStepRows) {
      s.sum[i] = sum;
      s.in[i] = in;
      s.leave[i] = (int16_t)leave;
      s.beta[i] = beta;
      s.grow[i] = expf((float)sum);
    }
  }
  bool before = false;  // chains: an earlier block holds a row that is no number
  for (int b = 0; b < blocks; ++b) {
    const int base = b * R, row0 = v.row0 + base, n = min(R, v.rows - base);
    if (b > 0) {
      __syncthreads();
      if (tid == 0) s.odd_q = 0;
      if (!chain && wave == 0) {
        const int lane = thread_now();
        const bool no = lane < R && ((s.in[base - R + min(lane, R - 1)] & s.odd[b - 1]) || s.behind[min(lane, R - 1)]);
        const unsigned long long all = __ballot(no);
        if (lane == 0) s.odd[b - 1] = all;
      }
      __syncthreads();
    }
    if (b > 0) fetch(b);
    keys.store(n, s.k, KS, &s.odd[b]);
    queries.store(n, s.q, KS, &s.odd_q);
    f32x4 rhs[RT];
    {
      const int lane = thread_now() & 63, g = lane >> 4;
      unsigned long long odd = 0;
#pragma unroll
      for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int i = 16 * m + 4 * g + r;
          const uint32_t x = values[m][r];
          const bool no = is_odd(odd_sum(x));
          if (no && i < n) odd |= 1ull << i;
          rhs[m][r] = no || i >= n ? 0.0f : __uint_as_float(x << 16);
        }
      if (odd) atomicOr(&s.odd[b], odd);
    }
    if (tid < R) s.behind[tid] = 0, s.next[tid] = base + tid < v.rows ? s.leave[base + tid] : -1;
    __syncthreads();
    if (s.bad) {
      if (!(s.bad & 2)) no_numbers(a, v, head, VD, vw - wave * 16, 16 * kWaves);
      return;
    }
    if (b > 0 && !chain) {  // sums from the state, now that those of the rows above the block are
      if (tid < n) {
        const int up = s.leave[base + tid];
        if (up >= 0) {
          const double sum = s.sum[base + tid] + s.sum[up];
          s.sum[base + tid] = sum;
          s.grow[base + tid] = expf((float)sum);
        }
      }
      __syncthreads();
    }

    // tiles of the block: diagonal ones of L first, each inverted by the wave that made it
    const auto tile = [&](bool of_low, int bi, int bj) {
      const int lane = thread_now() & 63, col = lane & 15, g = lane >> 4;
      f32x4 x = pair_tile<KD>((of_low ? s.k : s.q) + 16 * bi * KS, s.k + 16 * bj * KS, KS, lane);
      const int i = 16 * bi + col, at = base + i;
      const unsigned long long in = s.in[at];
      const double gi = s.sum[at];
      const float f = of_low ? -s.beta[at] : 1.0f;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = 16 * bj + 4 * g + r;
        const bool on = i < n && ((in >> j) & 1) && !(of_low && i == j);
        // (__expf: off by about |x| 2^-23 of itself, as much as its argument's rounding to fp32)
        x[r] = on ? f * __expf((float)(gi - s.sum[base + j])) * x[r] : 0.0f;
      }
      (of_low ? s.low : s.see)[bi * RT + bj][lane] = x;
    };
    // (a loop, as the code runs once and its instructions have to be fetched)
#pragma unroll 1
    for (int turn = 0, item = role; turn * kWaves < RT + RT * RT; ++turn) {
      if (item < RT) {
        tile(true, item, item);
        wave_lds_sync();
        invert<(RT > 1)>(s.low[item * RT + item], s.inv[item], n - 16 * item);
      } else if (item < RT + RT * RT) {
        const int i = (item - RT) / RT, j = (item - RT) % RT;
        tile(j > i, max(i, j), min(i, j));
      }
      item = (turn + 1) * kWaves + (turn & 1 ? role : kWaves - 1 - role);
    }

    // the rows' products with the old state
    f32x4 acc[RT];
    {
      const int lane = thread_now() & 63, col = lane & 15, g = lane >> 4;
      f32x4 w[RT];
#pragma unroll
      for (int m = 0; m < RT; ++m) w[m] = acc[m] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int t = 0; t < KT; t += 2) {
        uint4 piece[3];
        split3(S[t][0], S[t + 1][0], piece[0], piece[1], piece[2]);
#pragma unroll
        for (int m = 0; m < RT; ++m) {
          const uint4 fk = fragment(s.k + (16 * m + col) * KS + 16 * t + 4 * g);
          const uint4 fq = fragment(s.q + (16 * m + col) * KS + 16 * t + 4 * g);
#pragma unroll
          for (int p = 2; p >= 0; --p) {
            w[m] = mfma_bf16(fk, piece[p], w[m]);
            acc[m] = mfma_bf16(fq, piece[p], acc[m]);
          }
        }
      }
#pragma unroll
      for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int i = base + 16 * m + 4 * g + r;
          const float grow = s.grow[i], beta = s.beta[i];
          rhs[m][r] = i < v.rows ? beta * (rhs[m][r] - grow * w[m][r]) : 0.0f;
          acc[m][r] *= grow;
        }
    }

    // trees: the path's rows in earlier blocks, the nearest first
    if (!chain) {
      for (int e = b - 1; e >= 0; --e) {
        __syncthreads();
        const int lane = thread_now() & 63, col = lane & 15, g = lane >> 4, v0 = vw + col;
        keys.load(a.c.kv + kv_at(a.c, a.layer, v.row0 + e * R) + key * KD, a.c.kv_width, R);
        keys.store(R, s.t, KS, &s.odd[e]);
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
          f32x4 x = pair_tile<KD>((of_low ? s.k : s.q) + 16 * bi * KS, s.t + 16 * bj * KS, KS, lane);
          const unsigned long long in = s.cross[i];
          const double gi = s.sum[base + i];
          const float f = of_low ? -s.beta[base + i] : 1.0f;
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
          f32x4 d;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int j = 16 * mj + 4 * g + r;
            const float* p = deltas + ((uint32_t)j * hv * VD + v0);
            d[r] = (odd >> j) & 1 ? 0.0f : *p;
          }
#pragma unroll
          for (int m = 0; m < RT; ++m) {
            rhs[m] = mfma_f32(s.far_low[m * RT + mj][lane], d, rhs[m]);
            acc[m] = mfma_f32(s.far_see[m * RT + mj][lane], d, acc[m]);
          }
        }
      }
    }
    __syncthreads();

    // the triangular system, and the outputs
    const int lane = thread_now() & 63, col = lane & 15, g = lane >> 4, v0 = vw + col;
#pragma unroll
    for (int m = 0; m < RT; ++m) {
      f32x4 d = mfma_f32(s.inv[m][lane], rhs[m], f32x4{0, 0, 0, 0});
      rhs[m] = d;
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        if (i > m) rhs[i] = mfma_f32(s.low[i * RT + m][lane], d, rhs[i]);
        if (i >= m) acc[i] = mfma_f32(s.see[i * RT + m][lane], d, acc[i]);
      }
    }
    const unsigned long long odd = s.odd[b], odd_q = s.odd_q;
    uint16_t* outs = a.out + ((size_t)row0 * hv + head) * VD;
    float* deltas = a.c.delta + delta_at(a.c, a.layer, row0, head);
    const uint32_t step = hv * VD, at0 = 4 * g * step + v0;
    const bool plain = b == 0 && !odd && !odd_q;  // no row to set apart
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 16 * m + 4 * g + r;
        const uint32_t at = at0 + (16 * m + r) * step;
        uint16_t o = (uint16_t)bf16_pair(a.scale * acc[m][r], 0.0f);
        float d = rhs[m][r];
        if (!plain) {
          const bool no = before || (s.in[base + i] & odd) || (!chain && s.behind[i]);
          if (no || ((odd_q >> i) & 1)) o = 0x7FC0;
          if (no) d = __builtin_nanf("");
        }
        if (i < n) {
          *behind(outs, 2 * at) = o;
          if (!a.keep) *behind(deltas, 4 * at) = d;
        }
      }

    // chains: the state behind the block
    if constexpr (RT == 1) {
      before = before || (chain && odd);
      if (chain && (a.keep || b + 1 < blocks)) {
        // keys with rows innermost, and the decays to the block's end
        for (int e = thread_now(); e < 8 * (KD / 8); e += kThreads) {
          const int r = (e & 7) * 2, c = (e >> 3) * 8;
          store_turned(s.t + c * TS + r, TS, *reinterpret_cast<const uint4*>(s.k + r * KS + c),
                       *reinterpret_cast<const uint4*>(s.k + (r + 1) * KS + c));
        }
        if (tid < R) s.part[tid] = tid < n ? expf((float)(s.sum[base + n - 1] - s.sum[base + tid])) : 0.0f;
        __syncthreads();
        const float keep = s.grow[base + n - 1];
        uint4 piece[3];
        f32x4 y;
#pragma unroll
        for (int r = 0; r < 4; ++r) y[r] = s.part[4 * g + r] * rhs[0][r];
        split3(y, f32x4{0, 0, 0, 0}, piece[0], piece[1], piece[2]);
#pragma unroll
        for (int t = 0; t < KT; ++t) {
          const uint2 x = *reinterpret_cast<const uint2*>(s.t + (16 * t + col) * TS + 4 * g);
          const uint4 f = make_uint4(x.x, x.y, 0, 0);
          f32x4 add = {0, 0, 0, 0};
#pragma unroll
          for (int p = 2; p >= 0; --p) add = mfma_bf16(f, piece[p], add);
          join_state(S[t][0], keep, add);
        }
      }
    }
  }
  if (RT == 1 && a.keep) {
    if (before) {
#pragma unroll
      for (int t = 0; t < KT; ++t) S[t][0] = f32x4{__builtin_nanf(""), __builtin_nanf(""), __builtin_nanf(""), __builtin_nanf("")};
    }
    store_state<KT, VD, 1>(state, vw, S);
    keep_window(a, v);
  }
}

// Plain decoding: as many rows as sequences, chains. Two dims a lane of 128 x 128
// spill 8 registers at four waves a SIMD, none at three: 32 x 1 42.2 us against 41.8,
// 8 x 1 14.0 / 13.7, 64 x 1 76.8 / 77.0.
constexpr int kDecodeThreads = 256;
template <int KD, int VD, int NC>
__global__ __launch_bounds__(kDecodeThreads, 4) void delta_decode_kernel(DeltaRuleArgs a) {
  constexpr int kWaves = kDecodeThreads / 64;
  constexpr int KT = KD / 16, slabs = VD / (kWaves * 16 * NC);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int head = blockIdx.x / slabs, key = head / (a.c.value_heads / a.c.key_heads), seq = blockIdx.y;
  const int vw = (blockIdx.x - head * slabs) * (kWaves * 16 * NC) + wave * (16 * NC);
  const RowsView v = rows_view(a.c, a.st, seq);
  if (v.rows == 0) return;
  float* state = a.c.state + state_at(a.c, a.layer, v.slot, head);
  f32x4 S[KT][NC];
  const Look seen = look(a, v);
  load_state<KT, VD, NC>(state, vw, S);
  rows_in_turn<KD, VD, NC>(a, v, seq, head, key, vw, state, seen, S);
}

// Which form: by the rows a sequence has on average (their numbers are on the
// device) and by the workgroups there are. In us, 16 key and 48 value heads of
// 128 x 128 (other heads and dims go by their workgroups, not measured on both
// sides), sequences x rows, states rotated past the caches for single rows:
//   single rows, 32 value dims a wave (past the caches) against 16: 1 x 1 7.6 / 6.6,
//     2 x 1 7.8 / 7.1, 3 x 1 8.1 / 9.7, 8 x 1 14.0 / 17.8, 32 x 1 42.3 / 52.0.
//   trees, blocks of 16 / 32 / 64 rows: 24 x 8 24.0 / 38.2 / 99.9, 1 x 16 7.9 / 8.1 /
//     13.2, 1 x 24 13.9 / 8.5 / 13.5, 6 x 32 20.0 / 17.1 / 37.7, 1 x 64 32.9 / 17.7 / 15.2,
//     3 x 64 33.4 / 20.7 / 27.1 (a CU holds one workgroup of the last).
//   kept chains, delta_chain.hip against blocks of 16: 1 x 32 8.7 / 15.9, 1 x 64 10.8 /
//     27.0, 4 x 32 17.5 / 17.3, 6 x 32 25.7 / 22.7, 8 x 48 38.0 / 32.3, 8 x 64 37.1 / 39.8,
//     4 x 128 34.6 / 52.9, 16 x 32 57.7 / 40.5. Up to 16 rows all go in blocks of 16, for
//     two or fewer sequences the slower side: 1 x 8 8.9 / 9.2, 1 x 16 8.8 / 10.0, 2 x 16
//     9.9 / 10.6, but 3 x 16 17.7 / 10.9, 8 x 8 27.0 / 15.0, 8 x 16 28.0 / 16.2. Not kept:
//     1 x 32 6.8 / 13.4, 24 x 8 55.3 / 24.0, 8 x 48 30.0 / 28.8.
// A step's sequences need not be alike, and a long one among short ones is then
// in a form of the short ones' (right, and slow): 32 single kept rows and 480 of one
// sequence 185 to 210 us, where alone they take 40 and 44; 64 rows among 63 empty
// sequences 91 against 11, 512 among 511 empty ones 750 against 47; a tree of 400
// rows alone 271, with 24 single rows 303 to 337, with 40 of them 580. In two calls, the short
// sequences' rows first, they take 86 (chains), 291 and 298 (trees).
template <int KD, int VD>
hipError_t launch(const DeltaRuleArgs& a, hipStream_t s) {
  const int rows = (a.st.total + a.st.num_seq - 1) / a.st.num_seq;
  const int heads = a.c.value_heads * a.st.num_seq, groups = heads * (VD / 64);  // of 64 value dims
  const dim3 grid(a.c.value_heads * (VD / 64), a.st.num_seq), whole(a.c.value_heads, a.st.num_seq);
  if (rows == 1 && !a.st.parent) {
    if constexpr (VD == 128) {
      if (heads >= 128) {
        delta_decode_kernel<KD, VD, 2><<<whole, kDecodeThreads, 0, s>>>(a);
        return hipGetLastError();
      }
    }
    delta_decode_kernel<KD, VD, 1><<<grid, kDecodeThreads, 0, s>>>(a);
  } else if (rows <= 16 || (!a.st.parent && rows < 64 && groups > 384)) {
    delta_rule_kernel<KD, VD, 1, VD / 16><<<whole, VD * 4, 0, s>>>(a);
  } else if (!a.st.parent) {
    return launch_delta_chain(a, s);
  } else if (rows <= 32 || groups > 256) {
    delta_rule_kernel<KD, VD, 2, 4><<<grid, 256, 0, s>>>(a);
  } else {
    delta_rule_kernel<KD, VD, 4, 4><<<grid, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_rule(const DeltaRuleArgs& a, hipStream_t s) {
  if (a.c.key_dim == 64) return a.c.value_dim == 64 ? launch<64, 64>(a, s) : launch<64, 128>(a, s);
  return a.c.value_dim == 64 ? launch<128, 64>(a, s) : launch<128, 128>(a, s);
}

}  // namespace w12
