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
// logits); one workgroup per tree walks from the root; the next token is
// drawn from the last row, chunk sums over many workgroups, the last of a
// tree's to arrive finding the chunk and the token in it.
#include "kv_internal.h"
#include "w12_device.h"

namespace w12 {
namespace {

constexpr int kChunk = 4096;      // tokens of one workgroup of a row
constexpr int kStatThreads = 256;
constexpr int kWalkThreads = 1024;
constexpr int kTreeNodes = 1024;  // most nodes of a tree

struct Layout {
  int splits;
  size_t off_stat, off_sum, off_state, off_cnt, total;
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
  double max, sum, c;  // of the last row; c: the residual is max(p - c q, 0)
  int row, node;       // last row, -1: no token to draw; its node in the tree
  double pad;
};

__device__ __forceinline__ double logit(const SampledArgs& a, int row, int t) {
  const size_t at = (size_t)row * a.vocab + t;
  if (a.logits_f32) return (double)static_cast<const float*>(a.logits)[at];
  return (double)__uint_as_float((uint32_t)static_cast<const uint16_t*>(a.logits)[at] << 16);
}
__device__ __forceinline__ double inv_temperature(const SampledArgs& a, int tree) {
  return a.temperature ? 1.0 / (double)a.temperature[tree] : 1.0;
}

__device__ __forceinline__ double shfl_xor_d(double v, int o) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __shfl_xor((uint32_t)b, o, 64), hi = __shfl_xor((uint32_t)(b >> 32), o, 64);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
// Sum (maximum) over the workgroup in a fixed order, in every thread.
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
template <int NT>
__device__ __forceinline__ double block_max(double v, double* s_red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmax(v, shfl_xor_d(v, o));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s_red[threadIdx.x >> 6] = v;
  __syncthreads();
  double r = s_red[0];
#pragma unroll
  for (int i = 1; i < NT / 64; ++i) r = fmax(r, s_red[i]);
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
  __shared__ int s_tree;
  const int row = blockIdx.y, split = blockIdx.x, tid = threadIdx.x;
  const Layout L = layout_of(a.num_trees, a.total, a.vocab);
  char* ws = static_cast<char*>(a.ws);
  if (row == 0 && split == 0)
    for (int t = tid; t < a.num_trees; t += kStatThreads) reinterpret_cast<uint32_t*>(ws + L.off_cnt)[t] = 0;
  const int tree = tree_of<kStatThreads>(a, row, &s_tree);
  if (tree >= a.num_trees) return;
  const double it = inv_temperature(a, tree);
  const int t0 = split * kChunk;
  double x[kChunk / kStatThreads], mx = -__builtin_huge_val();
#pragma unroll
  for (int i = 0; i < kChunk / kStatThreads; ++i) {
    const int t = t0 + i * kStatThreads + tid;
    x[i] = t < a.vocab ? logit(a, row, t) * it : -__builtin_huge_val();
    mx = fmax(mx, x[i]);
  }
  mx = block_max<kStatThreads>(mx, s_red);
  double sum = 0.0;
  if (mx > -__builtin_huge_val()) {
#pragma unroll
    for (int i = 0; i < kChunk / kStatThreads; ++i) sum += exp(x[i] - mx);
  } else {
    // nothing but -inf and NaN: a NaN must still reach the row's sum
#pragma unroll
    for (int i = 0; i < kChunk / kStatThreads; ++i) sum += x[i] != x[i] ? x[i] : 0.0;
  }
  sum = block_sum<kStatThreads>(sum, s_red);
  if (tid == 0) reinterpret_cast<double2*>(ws + L.off_stat)[(size_t)row * L.splits + split] = make_double2(mx, sum);
}

// Maximum and sum of a whole row from its chunks, in every thread.
template <int NT>
__device__ __forceinline__ void row_stat(const double2* st, int splits, double* s_red, double& mx, double& sum) {
  mx = -__builtin_huge_val();
  for (int i = threadIdx.x; i < splits; i += NT) mx = fmax(mx, st[i].x);
  mx = block_max<NT>(mx, s_red);
  double s = 0.0;
  for (int i = threadIdx.x; i < splits; i += NT) {
    const double2 v = st[i];
    s += v.x > -__builtin_huge_val() ? v.y * exp(v.x - mx) : v.y;
  }
  sum = block_sum<NT>(s, s_red);
}

// One workgroup walks one tree.
__global__ __launch_bounds__(kWalkThreads) void sampled_walk_kernel(SampledArgs a) {
  __shared__ int s_parent[kTreeNodes], s_token[kTreeNodes], s_next[kTreeNodes], s_first[kTreeNodes];
  __shared__ double s_red[kWalkThreads / 64];
  __shared__ int s_bad;
  const int t = blockIdx.x, tid = threadIdx.x;
  const Layout L = layout_of(a.num_trees, a.total, a.vocab);
  char* ws = static_cast<char*>(a.ws);
  State* state = reinterpret_cast<State*>(ws + L.off_state) + t;
  const int b0 = a.node_off[t], b1 = a.node_off[t + 1];
  const bool range_ok = b0 >= 0 && b0 <= b1 && b1 <= a.total;
  const int n = range_ok ? b1 - b0 : 0;
  const double it = inv_temperature(a, t);
  if (tid == 0) s_bad = (n < 1 || n > kTreeNodes || !(it > 0.0 && it < __builtin_huge_val())) ? 1 : 0;
  __syncthreads();
  if (n <= kTreeNodes) {
    for (int i = tid; i < n; i += kWalkThreads) {
      const int p = a.parent[b0 + i], tok = a.token[b0 + i];
      s_parent[i] = p;
      s_token[i] = tok;
      if (i == 0 ? p != -1 : (p < 0 || p >= i || tok < 0 || tok >= a.vocab)) s_bad = 1;
    }
  }
  __syncthreads();
  bool bad = s_bad;
  int last = 0, len = -1;
  double mx = 0.0, sum = 0.0, c = 0.0;
  if (!bad) {
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
    int node = 0;
    while (node >= 0) {
      ++len;
      last = node;
      const int row = b0 + node;
      if (tid == 0) a.path[b0 + len] = node;
      row_stat<kWalkThreads>(reinterpret_cast<const double2*>(ws + L.off_stat) + (size_t)row * L.splits, L.splits, s_red, mx, sum);
      if (!(sum > 0.0 && sum < __builtin_huge_val())) {
        bad = true;
        break;
      }
      c = 0.0;
      double left = 1.0;  // n_r
      int chosen = -1;
      for (int k = s_first[node]; k >= 0; k = s_next[k]) {
        const int tok = s_token[k];
        const double p = exp(logit(a, row, tok) * it - mx) / sum;
        const double u = (double)a.u_accept[b0 + k];
        if (a.draft) {
          const float* q = a.draft + (size_t)row * a.vocab;
          const double qx = (double)q[tok];
          if (u * qx * left < p - c * qx) {
            chosen = k;
            break;
          }
          c += left;
          if (s_next[k] < 0) break;  // the draw sums its residual itself
          double r = 0.0;
          for (int i = tid; i < a.vocab; i += kWalkThreads)
            r += fmax(exp(logit(a, row, i) * it - mx) / sum - c * (double)q[i], 0.0);
          left = block_sum<kWalkThreads>(r, s_red);
        } else {
          bool again = false;
          for (int j = s_first[node]; j != k; j = s_next[j]) again = again || s_token[j] == tok;
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
    s.max = mx;
    s.sum = sum;
    s.c = c;
    s.row = bad ? -1 : b0 + last;
    s.node = last;
    *state = s;
  }
}

// The next token of each tree.
__global__ __launch_bounds__(kStatThreads) void sampled_draw_kernel(SampledArgs a) {
  constexpr int kPer = kChunk / kStatThreads;
  __shared__ double s_red[kStatThreads / 64];
  __shared__ double s_scan[kStatThreads];
  __shared__ uint32_t s_gone[kChunk / 32];
  __shared__ int s_last, s_chunk, s_pick, s_some;
  __shared__ double s_before;
  const int t = blockIdx.y, split = blockIdx.x, tid = threadIdx.x;
  const Layout L = layout_of(a.num_trees, a.total, a.vocab);
  char* ws = static_cast<char*>(a.ws);
  const State st = reinterpret_cast<const State*>(ws + L.off_state)[t];
  if (st.row < 0) return;
  const double it = inv_temperature(a, t);
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
  // (residual, p) of one token of the chunk
  auto weight = [&](int chunk, int k) {
    const int tok = chunk * kChunk + k;
    if (tok >= a.vocab) return make_double2(0.0, 0.0);
    const double p = exp(logit(a, st.row, tok) * it - st.max) / st.sum;
    if (a.draft) return make_double2(fmax(p - st.c * (double)a.draft[(size_t)st.row * a.vocab + tok], 0.0), p);
    return make_double2((s_gone[k >> 5] >> (k & 31)) & 1 ? 0.0 : p, p);
  };

  mark(split);
  double r = 0.0, p = 0.0;
  for (int i = 0; i < kPer; ++i) {
    const double2 w = weight(split, i * kStatThreads + tid);
    r += w.x;
    p += w.y;
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
    return __hip_atomic_load(residual ? &sums[i].x : &sums[i].y, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  };
  if (tid == 0) {
    double total = 0.0;
    bool residual = true;
    for (int i = 0; i < L.splits; ++i) total += sum_of(i, true);
    if (!(total > 0.0)) {  // nothing is left but by rounding: p itself
      residual = false;
      total = 0.0;
      for (int i = 0; i < L.splits; ++i) total += sum_of(i, false);
    }
    const double target = (double)a.u_bonus[t] * total;
    double before = 0.0, keep = 0.0;
    int chunk = -1, some = 0;
    for (int i = 0; i < L.splits; ++i) {
      const double v = sum_of(i, residual);
      if (v > 0.0) {
        chunk = i;  // at the end: the last chunk that holds anything
        keep = before;
        if (before + v > target) {
          some = 1;
          break;
        }
      }
      before += v;
    }
    s_chunk = chunk;
    s_before = some ? target - keep : __builtin_huge_val();
    s_some = residual ? 1 : 0;
    s_pick = kChunk;
  }
  __syncthreads();
  const int chunk = s_chunk;
  const double target = s_before;
  const bool residual = s_some;
  mark(chunk);
  double w[kPer], own = 0.0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const double2 v = weight(chunk, tid * kPer + i);
    w[i] = residual ? v.x : v.y;
    own += w[i];
  }
  s_scan[tid] = own;
  __syncthreads();
  for (int o = 1; o < kStatThreads; o <<= 1) {
    const double x = tid >= o ? s_scan[tid - o] : 0.0;
    __syncthreads();
    s_scan[tid] += x;
    __syncthreads();
  }
  double cum = tid ? s_scan[tid - 1] : 0.0;
  int pick = kChunk, end = -1;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    cum += w[i];
    if (w[i] > 0.0) {
      end = tid * kPer + i;
      if (pick == kChunk && cum > target) pick = end;
    }
  }
  if (tid == 0) s_some = -1;
  __syncthreads();
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
