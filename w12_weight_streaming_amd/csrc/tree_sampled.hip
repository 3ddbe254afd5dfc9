// Sampled tree verification (gfx950): drafted tokens against the target's
// probabilities, from given random numbers.
//
// poot-llm docs, speculative sampling: a drafted token x is accepted with
// probability min(1, p(x) / q(x)), otherwise the next token comes from the
// normalised max(0, p - q). On a tree the children of a node are tried in
// index order against what the rejections so far have left of p. After r
// rejections that is
//   p_r = max(p - c_r q, 0) / n_r,   c_0 = 0, n_0 = 1,
//   c_{r+1} = c_r + n_r,   n_{r+1} = sum_t max(p(t) - c_{r+1} q(t), 0),
// (by induction: max(p_r - q, 0) = max(p - (c_r + n_r) q, 0) / n_r), so no
// residual is ever stored: a row's state is two numbers. Without draft
// probabilities a drafted token is certain (q is one at it): a rejection
// takes the token out of p.
//
// Outputs are token ids: two evaluations agree unless a random number falls
// between their cumulative sums, so probabilities, sums and comparisons are
// held in 64 bits (at 152064 tokens and 32 bits every hundredth draw would
// differ; at 64 none in 10^9).
//
// Three launches: chunk maxima and sums of every row (bound by reading the
// logits and by 64-bit arithmetic in equal parts); one workgroup per tree
// walks from the root, every node's probability looked up beforehand; the
// next token is drawn from the last row, chunk sums over many workgroups, the
// last of a tree's to arrive finding the chunk and the token in it.
#include "kv_internal.h"
#include "w12_device.h"

namespace w12 {
namespace {

constexpr int kChunk = 4096;      // tokens of one workgroup of a row
constexpr int kStatThreads = 256;
constexpr int kWalkThreads = 1024;
constexpr int kTreeNodes = 1024;  // most nodes of a tree
constexpr int kPer = kChunk / kStatThreads;  // neighbouring tokens of a thread
static_assert(kPer == 16);

struct Layout {
  int splits;
  size_t off_stat, off_sum, off_state, off_cnt, total;  // in the workspace
};
__host__ __device__ __forceinline__ Layout layout_of(int num_trees, int total, int vocab) {
  Layout l;
  l.splits = (vocab + kChunk - 1) / kChunk;
  l.off_stat = 0;                                               // [total][splits] (max, sum)
  l.off_sum = l.off_stat + (size_t)total * l.splits * 16;       // [num_trees][splits] (residual, p)
  l.off_state = l.off_sum + (size_t)num_trees * l.splits * 16;  // [num_trees] State
  l.off_cnt = l.off_state + (size_t)num_trees * 48;
  l.total = l.off_cnt + (((size_t)num_trees * 4 + 15) & ~size_t(15));
  return l;
}

// Where a tree's walk ended.
struct State {
  double sum, c;  // of the last row; c: the residual is max(p - c q, 0)
  float max;
  int row, node;  // last row, -1: no token to draw; its node in the tree
  int pad[3];
};

__device__ __forceinline__ float logit(const SampledArgs& a, int row, int t) {
  const size_t at = (size_t)row * a.vocab + t;
  if (a.logits_f32) return static_cast<const float*>(a.logits)[at];
  return __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.logits)[at] << 16);
}
__device__ __forceinline__ double inv_temperature(const SampledArgs& a, int tree) {
  return a.temperature ? 1.0 / (double)a.temperature[tree] : 1.0;
}

// 16 neighbouring values of a row from t on, in 16-byte loads where every row
// begins on 16 bytes; `fill` past the end.
__device__ __forceinline__ bool vectors(const void* p, int elem, int vocab) {
  return ((reinterpret_cast<uintptr_t>(p) | ((uintptr_t)vocab * elem)) & 15) == 0;
}
__device__ __forceinline__ void load16(const float* p, bool vec, int vocab, int t, float fill, float (&x)[kPer]) {
  if (vec && t + kPer <= vocab) {
#pragma unroll
    for (int i = 0; i < kPer; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + t + i);
      x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = t + i < vocab ? p[t + i] : fill;
  }
}
__device__ __forceinline__ void load16(const uint16_t* p, bool vec, int vocab, int t, float fill, float (&x)[kPer]) {
  if (vec && t + kPer <= vocab) {
#pragma unroll
    for (int i = 0; i < kPer; i += 8) {
      const uint4 v = *reinterpret_cast<const uint4*>(p + t + i);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[i + 2 * j] = __uint_as_float(w[j] << 16);
        x[i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = t + i < vocab ? __uint_as_float((uint32_t)p[t + i] << 16) : fill;
  }
}
__device__ __forceinline__ void logits16(const SampledArgs& a, int row, int t, float (&x)[kPer]) {
  const float none = -__builtin_huge_valf();
  if (a.logits_f32)
    load16(static_cast<const float*>(a.logits) + (size_t)row * a.vocab, vectors(a.logits, 4, a.vocab), a.vocab, t, none, x);
  else
    load16(static_cast<const uint16_t*>(a.logits) + (size_t)row * a.vocab, vectors(a.logits, 2, a.vocab), a.vocab, t, none, x);
}
__device__ __forceinline__ void draft16(const SampledArgs& a, int row, int t, float (&x)[kPer]) {
  load16(a.draft + (size_t)row * a.vocab, vectors(a.draft, 4, a.vocab), a.vocab, t, 0.f, x);
}

constexpr double kLog2e = 1.442695040888963407359925;
// exp((x - max) / temperature) in 64 bits, it2 = log2(e) / temperature: 2^y =
// 2^n 2^f with |f| <= 1/2 for y = (x - max) it2 (0 exactly at the maximum, at
// any temperature). n comes from adding 1.5 2^52, whose low bits then hold it;
// 2^f is its Taylor series
// to the 11th power (0.3466^12 / 12! = 6e-15 relative); 2^n goes straight into
// the exponent. Below 2^-1000, and for -inf, 0. Plain 64-bit multiply-adds
// throughout: conversions, ldexp and the library's exp made this twice and
// three times as slow, and it bounds the first launch.
__device__ __forceinline__ double weight_of(float x, double mx, double it2) {
  const double y = ((double)x - mx) * it2;
  const double t = y + 0x1.8p52;
  const double f = y - (t - 0x1.8p52);
  double p = 0x1.e8cac7351bb25p-32;  // ln(2)^k / k!
  p = __builtin_fma(p, f, 0x1.e4cf5158b8ecap-28);
  p = __builtin_fma(p, f, 0x1.b5253d395e7c4p-24);
  p = __builtin_fma(p, f, 0x1.62c0223a5c824p-20);
  p = __builtin_fma(p, f, 0x1.ffcbfc588b0c7p-17);
  p = __builtin_fma(p, f, 0x1.430912f86c787p-13);
  p = __builtin_fma(p, f, 0x1.5d87fe78a6731p-10);
  p = __builtin_fma(p, f, 0x1.3b2ab6fba4e77p-7);
  p = __builtin_fma(p, f, 0x1.c6b08d704a0c0p-5);
  p = __builtin_fma(p, f, 0x1.ebfbdff82c58fp-3);
  p = __builtin_fma(p, f, 0x1.62e42fefa39efp-1);
  p = __builtin_fma(p, f, 1.0);
  const uint64_t b = __builtin_bit_cast(uint64_t, p);
  const uint32_t n = (uint32_t)__builtin_bit_cast(uint64_t, t);
  const bool gone = !(y > -1000.0);
  const uint32_t hi = gone ? 0u : (uint32_t)(b >> 32) + (n << 20), lo = gone ? 0u : (uint32_t)b;
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

__device__ __forceinline__ double shfl_xor_d(double v, int o) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __shfl_xor((uint32_t)b, o, 64), hi = __shfl_xor((uint32_t)(b >> 32), o, 64);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
// Sum over the workgroup in a fixed order, in every thread.
template <int NT>
__device__ __forceinline__ double block_sum(double v, double* s_red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += shfl_xor_d(v, o);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s_red[threadIdx.x >> 6] = v;
  __syncthreads();
  double r = 0.0;
#pragma unroll
  for (int i = 0; i < NT / 64; ++i) r += s_red[i];
  return r;
}
// Tree of a row; num_trees where none holds it.
template <int NT>
__device__ __forceinline__ int tree_of(const SampledArgs& a, int row, int* s_tree) {
  if (threadIdx.x == 0) *s_tree = a.num_trees;
  __syncthreads();
  for (int t = threadIdx.x; t < a.num_trees; t += NT)
    if (row >= a.node_off[t] && row < a.node_off[t + 1]) atomicMin(s_tree, t);
  __syncthreads();
  return *s_tree;
}

// (max, sum of exp(x - max)) of one chunk of one row.
__global__ __launch_bounds__(kStatThreads) void sampled_stat_kernel(SampledArgs a) {
  __shared__ double s_red[kStatThreads / 64];
  __shared__ float s_top[kStatThreads / 64];
  __shared__ int s_tree;
  const int row = blockIdx.y, split = blockIdx.x, tid = threadIdx.x;
  const Layout L = layout_of(a.num_trees, a.total, a.vocab);
  char* ws = static_cast<char*>(a.ws);
  if (row == 0 && split == 0)
    for (int t = tid; t < a.num_trees; t += kStatThreads) reinterpret_cast<uint32_t*>(ws + L.off_cnt)[t] = 0;
  const int tree = tree_of<kStatThreads>(a, row, &s_tree);
  if (tree >= a.num_trees) return;
  const double it2 = inv_temperature(a, tree) * kLog2e;
  float x[kPer], top = -__builtin_huge_valf();
  bool nan = false;
  logits16(a, row, split * kChunk + tid * kPer, x);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    top = fmaxf(top, x[i]);
    nan = nan || x[i] != x[i];
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
  if ((tid & 63) == 0) s_top[tid >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kStatThreads / 64; ++i) top = fmaxf(top, s_top[i]);
  // a NaN or +inf must reach the row's sum; nothing but -inf has no weight
  const double mx = top;
  double sum = nan || top == __builtin_huge_valf() ? __builtin_nan("") : 0.0;
  if (top > -__builtin_huge_valf() && top < __builtin_huge_valf()) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum += weight_of(x[i], mx, it2);
  }
  sum = block_sum<kStatThreads>(sum, s_red);
  if (tid == 0) reinterpret_cast<double2*>(ws + L.off_stat)[(size_t)row * L.splits + split] = make_double2(top, sum);
}

// Maximum and sum of a whole row from its chunks, by one wave.
__device__ __forceinline__ void row_stat(const double2* st, int splits, double it2, float& mx, double& sum) {
  const int lane = threadIdx.x & 63;
  float m = -__builtin_huge_valf();
  for (int i = lane; i < splits; i += 64) m = fmaxf(m, (float)st[i].x);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
  double s = 0.0;
  for (int i = lane; i < splits; i += 64) {
    const double2 v = st[i];
    s += v.x > -__builtin_huge_val() && v.x < __builtin_huge_val() ? v.y * weight_of((float)v.x, m, it2) : v.y;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += shfl_xor_d(s, o);
  mx = m;
  sum = s;
}

// One workgroup walks one tree. The rows' maxima and sums (a wave each) and
// the nodes' probabilities (a thread each) come first, so that the walk itself
// reads nothing but LDS, save where a drawn draft is rejected and has siblings.
__global__ __launch_bounds__(kWalkThreads) void sampled_walk_kernel(SampledArgs a) {
  __shared__ int s_parent[kTreeNodes], s_token[kTreeNodes], s_next[kTreeNodes], s_first[kTreeNodes];
  __shared__ float s_max[kTreeNodes], s_u[kTreeNodes], s_q[kTreeNodes];
  __shared__ double s_sum[kTreeNodes], s_p[kTreeNodes];
  __shared__ double s_red[kWalkThreads / 64];
  __shared__ int s_bad;
  const int t = blockIdx.x, tid = threadIdx.x;
  const Layout L = layout_of(a.num_trees, a.total, a.vocab);
  char* ws = static_cast<char*>(a.ws);
  State* state = reinterpret_cast<State*>(ws + L.off_state) + t;
  const int b0 = a.node_off[t], b1 = a.node_off[t + 1];
  const bool range_ok = b0 >= 0 && b0 <= b1 && b1 <= a.total;
  const int n = range_ok ? b1 - b0 : 0;
  const double it = inv_temperature(a, t), it2 = it * kLog2e;
  if (tid == 0) s_bad = (n < 1 || n > kTreeNodes || !(it > 0.0 && it < __builtin_huge_val())) ? 1 : 0;
  __syncthreads();
  if (n <= kTreeNodes) {
    for (int i = tid; i < n; i += kWalkThreads) {
      const int p = a.parent[b0 + i], tok = a.token[b0 + i];
      s_parent[i] = p;
      s_token[i] = tok;
      s_u[i] = a.u_accept[b0 + i];
      if (i == 0 ? p != -1 : (p < 0 || p >= i || tok < 0 || tok >= a.vocab)) s_bad = 1;
    }
  }
  __syncthreads();
  bool bad = s_bad;
  int last = 0, len = -1;
  double c = 0.0;
  if (!bad) {
    for (int i = tid >> 6; i < n; i += kWalkThreads / 64) {
      float mx;
      double sum;
      row_stat(reinterpret_cast<const double2*>(ws + L.off_stat) + (size_t)(b0 + i) * L.splits, L.splits, it2, mx, sum);
      if ((tid & 63) == 0) {
        s_max[i] = mx;
        s_sum[i] = sum;
      }
    }
    for (int i = tid; i < n; i += kWalkThreads) {
      int first = -1, next = -1;
      for (int j = n - 1; j > i; --j) {
        if (s_parent[j] == i) first = j;
        if (s_parent[j] == s_parent[i]) next = j;
      }
      s_first[i] = first;
      s_next[i] = i == 0 ? -1 : next;
    }
    __syncthreads();
    for (int i = tid + 1; i < n; i += kWalkThreads) {
      const int up = s_parent[i], row = b0 + up;
      s_p[i] = weight_of(logit(a, row, s_token[i]), s_max[up], it2) / s_sum[up];
      if (a.draft) s_q[i] = a.draft[(size_t)row * a.vocab + s_token[i]];
    }
    __syncthreads();
    int node = 0;
    while (node >= 0) {
      ++len;
      last = node;
      const int row = b0 + node;
      if (tid == 0) a.path[b0 + len] = node;
      const double sum = s_sum[node];
      if (!(sum > 0.0 && sum < __builtin_huge_val())) {
        bad = true;
        break;
      }
      c = 0.0;
      double left = 1.0;  // n_r
      int chosen = -1;
      for (int k = s_first[node]; k >= 0; k = s_next[k]) {
        const double p = s_p[k], u = (double)s_u[k];
        if (a.draft) {
          const double qx = (double)s_q[k];
          if (u * qx * left < p - c * qx) {
            chosen = k;
            break;
          }
          c += left;
          if (s_next[k] < 0) break;  // the draw sums its residual itself
          const double mx = s_max[node];
          const double inv = 1.0 / sum;
          double r = 0.0;
          for (int i = tid * kPer; i < a.vocab; i += kWalkThreads * kPer) {
            float x[kPer], q[kPer];
            logits16(a, row, i, x);
            draft16(a, row, i, q);
#pragma unroll
            for (int j = 0; j < kPer; ++j) r += fmax(weight_of(x[j], mx, it2) * inv - c * (double)q[j], 0.0);
          }
          left = block_sum<kWalkThreads>(r, s_red);
        } else {
          bool again = false;
          for (int j = s_first[node]; j != k; j = s_next[j]) again = again || s_token[j] == s_token[k];
          if (!again) {
            if (u * left < p) {
              chosen = k;
              break;
            }
            left -= p;
          }
        }
      }
      node = chosen;
    }
  }
  __syncthreads();
  if (bad) {
    if (range_ok)
      for (int i = tid; i < n; i += kWalkThreads) a.path[b0 + i] = -1;
  } else {
    for (int i = len + 1 + tid; i < n; i += kWalkThreads) a.path[b0 + i] = -1;
  }
  if (tid == 0) {
    a.accept_len[t] = bad ? -1 : len;
    if (bad) a.bonus[t] = -1;
    State s{};
    s.max = bad ? 0.f : s_max[last];
    s.sum = bad ? 0.0 : s_sum[last];
    s.c = c;
    s.row = bad ? -1 : b0 + last;
    s.node = last;
    *state = s;
  }
}

// The next token of each tree.
__global__ __launch_bounds__(kStatThreads) void sampled_draw_kernel(SampledArgs a) {
  __shared__ double s_red[kStatThreads / 64];
  __shared__ double s_scan[kStatThreads / 64];
  __shared__ uint32_t s_gone[kChunk / 32];
  __shared__ int s_last, s_chunk, s_pick, s_some;
  __shared__ double s_before;
  const int t = blockIdx.y, split = blockIdx.x, tid = threadIdx.x;
  const Layout L = layout_of(a.num_trees, a.total, a.vocab);
  char* ws = static_cast<char*>(a.ws);
  const State st = reinterpret_cast<const State*>(ws + L.off_state)[t];
  if (st.row < 0) return;
  const double it2 = inv_temperature(a, t) * kLog2e;
  double2* sums = reinterpret_cast<double2*>(ws + L.off_sum) + (size_t)t * L.splits;
  const int b0 = a.node_off[t], n = a.node_off[t + 1] - b0;

  // bits of the chunk's tokens that rejections took out
  auto mark = [&](int chunk) {
    for (int i = tid; i < kChunk / 32; i += kStatThreads) s_gone[i] = 0;
    __syncthreads();
    if (!a.draft)
      for (int i = tid; i < n; i += kStatThreads)
        if (i > 0 && a.parent[b0 + i] == st.node) {
          const int k = a.token[b0 + i] - chunk * kChunk;
          if (k >= 0 && k < kChunk) atomicOr(&s_gone[k >> 5], 1u << (k & 31));
        }
    __syncthreads();
  };
  // (residual, p) of the thread's tokens of a chunk; without drafts in units
  // of the likeliest token's
  const double inv = a.draft ? 1.0 / st.sum : 1.0, mx = st.max;
  auto weights = [&](int chunk, double (&res)[kPer], double (&all)[kPer]) {
    const int t0 = chunk * kChunk + tid * kPer;
    float x[kPer], q[kPer];
    logits16(a, st.row, t0, x);
    if (a.draft) draft16(a, st.row, t0, q);
    const uint32_t gone = s_gone[tid >> 1] >> (tid & 1 ? 16 : 0);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      all[i] = weight_of(x[i], mx, it2) * inv;
      res[i] = a.draft ? fmax(all[i] - st.c * (double)q[i], 0.0) : (gone >> i) & 1 ? 0.0 : all[i];
    }
  };

  mark(split);
  double r = 0.0, p = 0.0;
  {
    double res[kPer], all[kPer];
    weights(split, res, all);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      r += res[i];
      p += all[i];
    }
  }
  r = block_sum<kStatThreads>(r, s_red);
  p = block_sum<kStatThreads>(p, s_red);
  if (tid == 0) {
    __hip_atomic_store(&sums[split].x, r, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(&sums[split].y, p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(0);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    s_last = atomicAdd(reinterpret_cast<uint32_t*>(ws + L.off_cnt) + t, 1u) == (uint32_t)(L.splits - 1) ? 1 : 0;
  }
  __syncthreads();
  if (!s_last) return;

  auto sum_of = [&](int i, bool residual) {
    if (i >= L.splits) return 0.0;
    return __hip_atomic_load(residual ? &sums[i].x : &sums[i].y, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  };
  // inclusive running sum over the threads; `whole`: over all of them
  auto running = [&](double v, double& whole) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint64_t w = __builtin_bit_cast(uint64_t, v);
      const uint32_t lo = __shfl_up((uint32_t)w, o, 64), hi = __shfl_up((uint32_t)(w >> 32), o, 64);
      if ((tid & 63) >= o) v += __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
    }
    __syncthreads();
    if ((tid & 63) == 63) s_scan[tid >> 6] = v;
    __syncthreads();
    whole = 0.0;
#pragma unroll
    for (int w = 0; w < kStatThreads / 64; ++w) {
      if (w < (tid >> 6)) v += s_scan[w];
      whole += s_scan[w];
    }
    return v;
  };
  double total = 0.0;
  for (int i = tid; i < L.splits; i += kStatThreads) total += sum_of(i, true);
  total = block_sum<kStatThreads>(total, s_red);
  const bool residual = total > 0.0;
  if (!residual) {  // nothing is left but by rounding: p itself
    total = 0.0;
    for (int i = tid; i < L.splits; i += kStatThreads) total += sum_of(i, false);
    total = block_sum<kStatThreads>(total, s_red);
  }
  // the first chunk in which the running sum passes the target; else the last
  // that holds anything, and in it the last token
  const double target = (double)a.u_bonus[t] * total;
  if (tid == 0) {
    s_chunk = L.splits;
    s_last = -1;
  }
  __syncthreads();
  double before = 0.0;
  for (int i0 = 0; i0 < L.splits; i0 += kStatThreads) {
    const double v = sum_of(i0 + tid, residual);
    double whole;
    const double upto = before + running(v, whole);
    if (v > 0.0) {
      atomicMax(&s_last, i0 + tid);
      if (upto > target) atomicMin(&s_chunk, i0 + tid);
    }
    __syncthreads();
    if (s_chunk == i0 + tid) s_before = target - (upto - v);
    __syncthreads();
    if (s_chunk < L.splits) break;
    before += whole;
  }
  if (tid == 0) {
    if (s_chunk == L.splits) {
      s_chunk = s_last;
      s_before = __builtin_huge_val();
    }
    s_pick = kChunk;
    s_some = -1;
  }
  __syncthreads();
  const int chunk = s_chunk;
  const double in_chunk = s_before;
  mark(chunk);
  double res[kPer], all[kPer], own = 0.0, whole;
  weights(chunk, res, all);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (!residual) res[i] = all[i];
    own += res[i];
  }
  double cum = running(own, whole) - own;
  int pick = kChunk, end = -1;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    cum += res[i];
    if (res[i] > 0.0) {
      end = tid * kPer + i;
      if (pick == kChunk && cum > in_chunk) pick = end;
    }
  }
  if (pick < kChunk) atomicMin(&s_pick, pick);
  if (end >= 0) atomicMax(&s_some, end);
  __syncthreads();
  if (tid == 0) a.bonus[t] = chunk * kChunk + (s_pick < kChunk ? s_pick : s_some);
}

}  // namespace

size_t tree_sampled_ws_bytes(int num_trees, int total, int vocab) { return layout_of(num_trees, total, vocab).total; }

hipError_t launch_tree_sampled(const SampledArgs& a, hipStream_t s) {
  const int splits = (a.vocab + kChunk - 1) / kChunk;
  hipLaunchKernelGGL(sampled_stat_kernel, dim3(splits, a.total), dim3(kStatThreads), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(sampled_walk_kernel, dim3(a.num_trees), dim3(kWalkThreads), 0, s, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(sampled_draw_kernel, dim3(splits, a.num_trees), dim3(kStatThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace w12
