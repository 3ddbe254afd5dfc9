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
// differ; at 64 fewer than one in 10^9).
//
// Two or three launches. Every wave takes the maximum and sum of a chunk of
// 1024 tokens (bound by its 64-bit arithmetic: vector instructions take 76% of a
// SIMD's time at 192 rows of 152064). One workgroup per tree walks from the root,
// every node's probability looked up beforehand, and, without draft
// probabilities, draws the next token: the chunks' sums are at hand, those that
// hold a rejected token are summed again without it. With draft probabilities
// every rejection that leaves siblings to try is a pass of that workgroup over
// the row (a branching tree of 32 nodes, 152064 tokens: 24 and 56 us a call at two
// random draws, 144 with nearly all drafts rejected), and the residual's chunk
// sums take another pass over the last row, by many workgroups; a tree's last to
// arrive finds the token.
#include "kv_internal.h"
#include "w12_device.h"

namespace w12 {
namespace {

constexpr int kChunk = 1024;   // tokens of a wave
constexpr int kPer = 16;       // neighbouring tokens of a lane
constexpr int kThreads = 256;  // of the launches over chunks: four chunks a workgroup
constexpr int kWaves = kThreads / 64;
constexpr int kTreeNodes = 1024;  // most nodes of a tree

// Where a tree's walk ended.
struct alignas(16) State {
  double sum, c;  // of the last row; c: the residual is max(p - c q, 0)
  float max;
  int row;  // last row, -1: no token to draw
};

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
  l.off_cnt = l.off_state + (size_t)num_trees * sizeof(State);
  l.total = l.off_cnt + (((size_t)num_trees * 4 + 15) & ~size_t(15));
  return l;
}

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
constexpr int kTable = 128, kTableLog = 7;
// exp((x - max) / temperature) in 64 bits: 2^(y / 128) = 2^(n / 128) 2^(f / 128)
// with |f| <= 1/2 for y = 128 (x - max) it2, it2 = log2(e) / temperature (0
// exactly at the maximum, at any temperature). n comes from adding 1.5 2^52,
// whose low bits then hold it: 2^(n mod 128 / 128) from a table in LDS, the rest
// of n straight into the exponent. 2^(f / 128) is its Taylor series to the 4th
// power: 1.2e-15 relative; with the table's and the argument's roundings 1.7e-15
// at the maximum, 2.7e-15 at e^-8, 8.6e-15 at e^-40 (4 million points each, against
// 80 bits). Below 2^-1000, and for -inf, 0.
// 64-bit arithmetic bounds the first launch: 192 rows of 152064 bf16 logits (58
// MB, 10 us of reading) take 52 us with the library's exp, 33 with a series to
// the 11th power and no table, 30 with 32 entries, the 5th power and separate
// products and sums, 27 like this.
struct Weigher {
  const double* table;  // LDS, kTable entries
  double mx, rate;
  float least, finite;  // logits at or below `least` (itself below the maximum) weigh nothing
  __device__ __forceinline__ Weigher(const double* t, float top, double it2) : table(t), mx(top), rate(kTable * it2) {
    least = fminf((float)(mx - 1000.0 / it2), nextafterf(top, -__builtin_huge_valf()));
    finite = fmaxf(least, -3.402823466e38f);
  }
  // n and the series of an x that is not below `finite` (others: any finite value)
  __device__ __forceinline__ double series(float x, int32_t& n) const {
    const double d = (double)x - mx;
    const double t = __builtin_fma(d, rate, 0x1.8p52);
    const double f = __builtin_fma(d, rate, 0x1.8p52 - t);
    double p = 0x1.3b2ab6fba4e77p-35;  // (ln(2) / 128)^k / k!
    p = __builtin_fma(p, f, 0x1.c6b08d704a0c0p-26);
    p = __builtin_fma(p, f, 0x1.ebfbdff82c58fp-17);
    p = __builtin_fma(p, f, 0x1.62e42fefa39efp-8);
    p = __builtin_fma(p, f, 1.0);
    n = (int32_t)__builtin_bit_cast(uint64_t, t);
    return p;
  }
  // the power of two that goes with it, as its halves
  __device__ __forceinline__ void power(int32_t n, uint32_t& hi, uint32_t& lo) const {
    const uint64_t b = __builtin_bit_cast(uint64_t, table[n & (kTable - 1)]);
    hi = (uint32_t)(b >> 32) + ((uint32_t)(n & -kTable) << (20 - kTableLog));
    lo = (uint32_t)b;
  }
  __device__ __forceinline__ double operator()(float x) const {
    int32_t n;
    uint32_t hi, lo;
    const double p = series(fmaxf(x, finite), n);
    power(n, hi, lo);
    const bool some = x > least;
    return p * __builtin_bit_cast(double, ((uint64_t)(some ? hi : 0u) << 32) | (some ? lo : 0u));
  }
  // Sum of N weights, the maximum's 1 among them. What lies 500 powers of two
  // below it may then count as just that (a clamp in place of two selects an
  // element), if the logits are fine enough for such a value and reach so far.
  template <int N>
  __device__ __forceinline__ double sum(const float (&x)[N]) const {
    const float low = (float)(mx - 500.0 * kTable / rate);
    const double depth = (mx - (double)low) * rate;
    double r = 0.0;
    if (depth > 200.0 * kTable && depth < 1000.0 * kTable) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        int32_t n;
        uint32_t hi, lo;
        const double p = series(__builtin_amdgcn_fmed3f(x[i], low, __builtin_huge_valf()), n);
        power(n, hi, lo);
        r = __builtin_fma(p, __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo), r);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) r += (*this)(x[i]);
    }
    return r;
  }
};
__device__ const double kPowers[32] = {
    0x1.0000000000000p+0, 0x1.059b0d3158574p+0, 0x1.0b5586cf9890fp+0, 0x1.11301d0125b51p+0,
    0x1.172b83c7d517bp+0, 0x1.1d4873168b9aap+0, 0x1.2387a6e756238p+0, 0x1.29e9df51fdee1p+0,
    0x1.306fe0a31b715p+0, 0x1.371a7373aa9cbp+0, 0x1.3dea64c123422p+0, 0x1.44e086061892dp+0,
    0x1.4bfdad5362a27p+0, 0x1.5342b569d4f82p+0, 0x1.5ab07dd485429p+0, 0x1.6247eb03a5585p+0,
    0x1.6a09e667f3bcdp+0, 0x1.71f75e8ec5f74p+0, 0x1.7a11473eb0187p+0, 0x1.82589994cce13p+0,
    0x1.8ace5422aa0dbp+0, 0x1.93737b0cdc5e5p+0, 0x1.9c49182a3f090p+0, 0x1.a5503b23e255dp+0,
    0x1.ae89f995ad3adp+0, 0x1.b7f76f2fb5e47p+0, 0x1.c199bdd85529cp+0, 0x1.cb720dcef9069p+0,
    0x1.d5818dcfba487p+0, 0x1.dfc97337b9b5fp+0, 0x1.ea4afa2a490dap+0, 0x1.f50765b6e4540p+0,
};
__device__ const double kFine[4] = {0x1.0000000000000p+0, 0x1.0163da9fb3335p+0, 0x1.02c9a3e778061p+0, 0x1.04315e86e7f85p+0};  // 2^(k / 128)
// The table in LDS, a product of the two above; the caller synchronises before its first use.
__device__ __forceinline__ void load_powers(double* s_pow) {
  if (threadIdx.x < kTable) s_pow[threadIdx.x] = kPowers[threadIdx.x / 4] * kFine[threadIdx.x % 4];
}

// A lane's value from 1, 2, 4 or 8 lanes before it in its row of 16 (around).
template <int N>
__device__ __forceinline__ uint32_t from_row(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xF, 0xF, false);
}
template <int N>
__device__ __forceinline__ double from_row(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = from_row<N>((uint32_t)b), hi = from_row<N>((uint32_t)(b >> 32));
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double lane_of(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)b, lane), hi = __builtin_amdgcn_readlane((uint32_t)(b >> 32), lane);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
// Sum (maximum) over the wave in a fixed order, the same in every lane: rows
// of 16 by lane moves, then the four rows' first lanes.
__device__ __forceinline__ double wave_sum(double v) {
  v += from_row<8>(v);
  v += from_row<4>(v);
  v += from_row<2>(v);
  v += from_row<1>(v);
  return (lane_of(v, 0) + lane_of(v, 16)) + (lane_of(v, 32) + lane_of(v, 48));
}
__device__ __forceinline__ float wave_max(float v) {
  auto step = [](float x, uint32_t y) { return fmaxf(x, __uint_as_float(y)); };
  v = step(v, from_row<8>(__float_as_uint(v)));
  v = step(v, from_row<4>(__float_as_uint(v)));
  v = step(v, from_row<2>(__float_as_uint(v)));
  v = step(v, from_row<1>(__float_as_uint(v)));
  auto at = [v](int lane) { return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane)); };
  return fmaxf(fmaxf(at(0), at(16)), fmaxf(at(32), at(48)));
}

// Sum over the workgroup in a fixed order, in every thread.
template <int NT>
__device__ __forceinline__ double block_sum(double v, double* s_red) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s_red[threadIdx.x >> 6] = v;
  __syncthreads();
  double r = 0.0;
#pragma unroll
  for (int i = 0; i < NT / 64; ++i) r += s_red[i];
  return r;
}
// Inclusive running sum over the workgroup's threads; `whole`: over all.
template <int NT>
__device__ __forceinline__ double running_sum(double v, double* s_scan, double& whole) {
  const int tid = threadIdx.x;
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
  for (int w = 0; w < NT / 64; ++w) {
    if (w < (tid >> 6)) v += s_scan[w];
    whole += s_scan[w];
  }
  return v;
}

// What the threads of a workgroup found, one entry a wave. Lanes are told apart
// by ballots: LDS atomics on one address with a value a lane run lane by lane (a
// search took 5 us with them, under 1 so).
template <int NT>
struct Search {
  int first[NT / 64], last[NT / 64];
  double rest[NT / 64];
};
constexpr int kNone = 1 << 30;
// The least `first` and the greatest `last` over the workgroup; both grow with the
// thread (kNone, -1: none), and `rest` belongs to `first`.
template <int NT>
__device__ __forceinline__ void search_join(int& first, int& last, double& rest, Search<NT>& s) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint64_t has = __ballot(first != kNone), any = __ballot(last >= 0);
  if (lane == (has ? __builtin_ctzll(has) : 0)) {
    s.first[wave] = first;
    s.rest[wave] = rest;
  }
  if (lane == (any ? 63 - __builtin_clzll(any) : 0)) s.last[wave] = last;
  __syncthreads();
  first = kNone;
  last = -1;
#pragma unroll
  for (int w = NT / 64 - 1; w >= 0; --w) {
    if (s.first[w] != kNone) {
      first = s.first[w];
      rest = s.rest[w];
    }
    if (last < 0) last = s.last[w];
  }
  __syncthreads();
}

// The first of `splits` chunks, value(i) each, at which the running sum passes
// `target`, and what of the target is left in it; else the last chunk that
// holds anything, with an infinite rest.
struct Found {
  int chunk;
  double rest;
};
template <int NT, typename F>
__device__ __forceinline__ Found find_chunk(F value, int splits, double target, double* s_scan, Search<NT>& s) {
  const int tid = threadIdx.x;
  double before = 0.0;
  Found f{0, __builtin_huge_val()};
  for (int i0 = 0; i0 < splits; i0 += NT) {
    const int i = i0 + tid;
    const double v = i < splits ? value(i) : 0.0;
    double whole;
    const double upto = before + running_sum<NT>(v, s_scan, whole);
    int first = v > 0.0 && upto > target ? i : kNone, last = v > 0.0 ? i : -1;
    double rest = target - (upto - v);
    search_join<NT>(first, last, rest, s);
    if (first != kNone) {
      f.chunk = first;
      f.rest = rest;
      break;
    }
    if (last >= 0) f.chunk = last;
    before += whole;
  }
  return f;
}
// The first of N tokens a thread (weights w, in order over the threads) at
// which the running sum passes `rest`; else the last with any weight.
template <int NT, int N>
__device__ __forceinline__ int find_token(const double (&w)[N], double rest, double* s_scan, Search<NT>& s) {
  const int tid = threadIdx.x;
  double own = 0.0, whole;
#pragma unroll
  for (int i = 0; i < N; ++i) own += w[i];
  double cum = running_sum<NT>(own, s_scan, whole) - own;
  int first = kNone, last = -1;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    cum += w[i];
    if (w[i] > 0.0) {
      last = tid * N + i;
      if (first == kNone && cum > rest) first = last;
    }
  }
  search_join<NT>(first, last, rest, s);
  return first != kNone ? first : last;
}

// (max, sum of exp(x - max)) of chunks of a row: `each` neighbouring ones a
// wave, the next one's logits on their way while one is summed.
__global__ __launch_bounds__(kThreads) void sampled_stat_kernel(SampledArgs a, int each) {
  const int row = blockIdx.y, lane = threadIdx.x & 63;
  const Layout L = layout_of(a.num_trees, a.total, a.vocab);
  const int first = (blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * each;
  const int end = min(first + each, L.splits);
  char* ws = static_cast<char*>(a.ws);
  if (row == 0 && blockIdx.x == 0)
    for (int t = threadIdx.x; t < a.num_trees; t += kThreads) reinterpret_cast<uint32_t*>(ws + L.off_cnt)[t] = 0;
  __shared__ double s_pow[kTable];
  load_powers(s_pow);
  float x[kPer], next[kPer];
  if (first < end) logits16(a, row, first * kChunk + lane * kPer, x);
  __syncthreads();
  if (first >= end) return;
  int tree = -1;  // the first that holds the row
  for (int t = 0; t < a.num_trees && tree < 0; t += 64) {
    const bool in = t + lane < a.num_trees && rows_meet(a.node_off, a.total, t + lane, row, 1);
    const uint64_t hit = __ballot(in);
    if (hit) tree = t + __builtin_ctzll(hit);
  }
  if (tree < 0) return;
  const double it2 = inv_temperature(a, tree) * kLog2e;
  for (int split = first; split < end; ++split) {
    if (split + 1 < end) logits16(a, row, (split + 1) * kChunk + lane * kPer, next);
    float top = -__builtin_huge_valf();
    bool nan = false;
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
      top = fmaxf(fmaxf(top, x[i]), x[i + 1]);
      nan = nan || __builtin_isunordered(x[i], x[i + 1]);
    }
    top = wave_max(top);
    // a NaN or +inf must reach the row's sum; nothing but -inf has no weight
    double sum = nan || top == __builtin_huge_valf() ? __builtin_nan("") : 0.0;
    if (top > -__builtin_huge_valf() && top < __builtin_huge_valf()) {
      sum += Weigher(s_pow, top, it2).sum(x);
    }
    sum = wave_sum(sum);
    if (lane == 0) reinterpret_cast<double2*>(ws + L.off_stat)[(size_t)row * L.splits + split] = make_double2(top, sum);
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = next[i];
  }
}

// Maximum and sum of a whole row from its chunks, by one wave: up to 256
// chunks (262144 tokens) stay in its registers, so they are read once.
__device__ __forceinline__ void row_stat(const double2* st, int splits, const double* s_pow, double it2, float& mx, double& sum) {
  constexpr int kKeep = 4;
  const int lane = threadIdx.x & 63;
  const double none = -__builtin_huge_val();
  double2 v[kKeep];
#pragma unroll
  for (int i = 0; i < kKeep; ++i) v[i] = lane + i * 64 < splits ? st[lane + i * 64] : make_double2(none, 0.0);
  float m = -__builtin_huge_valf();
#pragma unroll
  for (int i = 0; i < kKeep; ++i) m = fmaxf(m, (float)v[i].x);
  for (int i = lane + kKeep * 64; i < splits; i += 64) m = fmaxf(m, (float)st[i].x);
  m = wave_max(m);
  double s = 0.0;
  const Weigher weigh(s_pow, m, it2);
  auto add = [&](const double2 c) { s += c.x > none && c.x < -none ? c.y * weigh((float)c.x) : c.y; };
#pragma unroll
  for (int i = 0; i < kKeep; ++i) add(v[i]);
  for (int i = lane + kKeep * 64; i < splits; i += 64) add(st[i]);
  mx = m;
  sum = wave_sum(s);
}

// One workgroup walks one tree. The rows' maxima and sums (a wave each) and
// the nodes' probabilities (a thread each) come first, so that the walk itself
// reads nothing but LDS, save where a drawn draft is rejected and has siblings
// (a pass over the row: these trees get 1024 threads, the others 256). Bound by
// its chain of dependent loads: 14 us for 24 trees of 8 nodes.
template <int NT>
__global__ __launch_bounds__(NT) void sampled_walk_kernel(SampledArgs a) {
  constexpr int kWalkThreads = NT;
  __shared__ double s_pow[kTable];
  load_powers(s_pow);
  __shared__ int s_parent[kTreeNodes], s_token[kTreeNodes], s_next[kTreeNodes], s_first[kTreeNodes];
  __shared__ float s_max[kTreeNodes], s_u[kTreeNodes], s_q[kTreeNodes];
  __shared__ double s_sum[kTreeNodes], s_p[kTreeNodes];
  __shared__ double s_red[kWalkThreads / 64], s_fix[kTreeNodes];
  __shared__ Search<NT> s_search;
  __shared__ uint32_t s_gone[kWalkThreads / 64][kChunk / 32];
  __shared__ int s_bad, s_kids;
  const int t = blockIdx.x, tid = threadIdx.x;
  const Layout L = layout_of(a.num_trees, a.total, a.vocab);
  char* ws = static_cast<char*>(a.ws);
  State* state = reinterpret_cast<State*>(ws + L.off_state) + t;
  const int b0 = a.node_off[t], b1 = a.node_off[t + 1];
  bool range_ok = b0 >= 0 && b0 <= b1 && b1 <= a.total;
  int meets = 0;
  if (range_ok)
    for (int j = tid; j < t; j += kWalkThreads) meets |= rows_meet(a.node_off, a.total, j, b0, b1 - b0);
  range_ok = !__syncthreads_or(meets) && range_ok;
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
    // on its way while the rows are summed
    const float first_logit = tid + 1 < n ? logit(a, b0 + s_parent[tid + 1], s_token[tid + 1]) : 0.f;
    for (int i = tid >> 6; i < n; i += kWalkThreads / 64) {
      float mx;
      double sum;
      row_stat(reinterpret_cast<const double2*>(ws + L.off_stat) + (size_t)(b0 + i) * L.splits, L.splits, s_pow, it2, mx, sum);
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
      if (!a.draft) {  // a token that an earlier sibling's rejection takes out of p: nothing is left of it
        const int up = s_parent[i], tok = s_token[i];
        int again = 0;
#pragma unroll 4
        for (int j = 1; j < i; ++j) again |= (s_parent[j] == up) & (s_token[j] == tok);
        s_q[i] = again ? 0.f : 1.f;
      }
    }
    __syncthreads();
    for (int i = tid + 1; i < n; i += kWalkThreads) {
      const int up = s_parent[i], row = b0 + up;
      s_p[i] = Weigher(s_pow, s_max[up], it2)(i == tid + 1 ? first_logit : logit(a, row, s_token[i])) / s_sum[up];
      if (a.draft)
        s_q[i] = a.draft[(size_t)row * a.vocab + s_token[i]];
      else if (s_q[i] == 0.f)
        s_p[i] = 0.0;
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
          const Weigher weigh(s_pow, s_max[node], it2);
          const double inv = 1.0 / sum;
          double r = 0.0;
          for (int i = tid * kPer; i < a.vocab; i += kWalkThreads * kPer) {
            float x[kPer], q[kPer];
            logits16(a, row, i, x);
            draft16(a, row, i, q);
#pragma unroll
            for (int j = 0; j < kPer; ++j) r += fmax(weigh(x[j]) * inv - c * (double)q[j], 0.0);
          }
          left = block_sum<kWalkThreads>(r, s_red);
        } else {
          if (p > 0.0 && u * left < p) {
            chosen = k;
            break;
          }
          left -= p;
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
    if (a.draft) {
      State s{};
      s.max = bad ? 0.f : s_max[last];
      s.sum = bad ? 0.0 : s_sum[last];
      s.c = c;
      s.row = bad ? -1 : b0 + last;
      *state = s;
    }
    s_kids = 0;
  }
  if (bad || a.draft) return;

  // The next token, of the last row without its children's tokens.
  const int row = b0 + last;
  const Weigher weigh(s_pow, s_max[last], it2);
  const double2* st = reinterpret_cast<const double2*>(ws + L.off_stat) + (size_t)row * L.splits;
  int* s_list = s_next;  // the children, in no order (the walk is done)
  __syncthreads();
  for (int i = tid + 1; i < n; i += kWalkThreads)
    if (s_parent[i] == last) s_list[atomicAdd(&s_kids, 1)] = s_token[i];
  __syncthreads();
  const int kids = s_kids, wave = tid >> 6, lane = tid & 63;
  auto mark = [&](uint32_t* gone, int chunk, int first, int step) {
    for (int k = first; k < kids; k += step) {
      const int j = s_list[k] - chunk * kChunk;
      if (j >= 0 && j < kChunk) atomicOr(&gone[j >> 5], 1u << (j & 31));
    }
  };
  // chunks with a child's token, summed anew by a wave each, for the first of
  // their children on the list
  for (int k = wave; k < kids; k += kWalkThreads / 64) {
    const int chunk = s_list[k] / kChunk;
    bool done = false;
    for (int j = lane; j < k; j += 64) done = done || s_list[j] / kChunk == chunk;
    if (__any(done)) continue;
    uint32_t* gone = s_gone[wave];
    if (lane < kChunk / 32) gone[lane] = 0;
    wave_lds_sync();
    mark(gone, chunk, lane, 64);
    wave_lds_sync();
    float x[kPer];
    logits16(a, row, chunk * kChunk + lane * kPer, x);
    const uint32_t out = gone[lane >> 1] >> (lane & 1 ? 16 : 0);
    double r = 0.0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) r += (out >> i) & 1 ? 0.0 : weigh(x[i]);
    r = wave_sum(r);
    if (lane == 0) s_fix[k] = r;
    wave_lds_sync();
  }
  __syncthreads();
  bool taken = true;  // the children's tokens are out (unless nothing else is left)
  auto chunk_sum = [&](int i) {
    const double2 v = st[i];
    double r = v.x > -__builtin_huge_val() ? v.y * weigh((float)v.x) : 0.0;
    if (taken)
      for (int k = 0; k < kids; ++k)
        if (s_list[k] / kChunk == i) {
          r = s_fix[k];
          break;
        }
    return r;
  };
  double total = 0.0;
  for (int i = tid; i < L.splits; i += kWalkThreads) total += chunk_sum(i);
  total = block_sum<kWalkThreads>(total, s_red);
  if (!(total > 0.0)) {  // by rounding only: p itself
    taken = false;
    total = 0.0;
    for (int i = tid; i < L.splits; i += kWalkThreads) total += chunk_sum(i);
    total = block_sum<kWalkThreads>(total, s_red);
  }
  const Found f = find_chunk<kWalkThreads>(chunk_sum, L.splits, (double)a.u_bonus[t] * total, s_red, s_search);
  if (tid < kChunk / 32) s_gone[0][tid] = 0;
  __syncthreads();
  if (taken) mark(s_gone[0], f.chunk, tid, kWalkThreads);
  __syncthreads();
  constexpr int N = kChunk / NT;
  double w[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int j = tid * N + i, tok = f.chunk * kChunk + j;
    w[i] = tok < a.vocab && !((s_gone[0][j >> 5] >> (j & 31)) & 1) ? weigh(logit(a, row, tok)) : 0.0;
  }
  const int pick = find_token<NT>(w, f.rest, s_red, s_search);
  if (tid == 0) a.bonus[t] = f.chunk * kChunk + pick;
}

// The next token of each tree whose drafts were drawn: from the last row's
// max(p - c q, 0), or from p where nothing of that is left (by rounding). A walk
// that ends at a node without children has c = 0 (others at least 1): its row of
// q is not read, so what it holds, NaN or infinities (0 inf = NaN) too, takes no weight.
__global__ __launch_bounds__(kThreads) void sampled_draw_kernel(SampledArgs a) {
  __shared__ double s_red[kWaves], s_pow[kTable];
  __shared__ Search<kThreads> s_search;
  __shared__ int s_last;
  const int t = blockIdx.y, tid = threadIdx.x, lane = tid & 63;
  const int split = blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(tid >> 6);
  const Layout L = layout_of(a.num_trees, a.total, a.vocab);
  char* ws = static_cast<char*>(a.ws);
  const State st = reinterpret_cast<const State*>(ws + L.off_state)[t];
  if (st.row < 0) return;
  const double it2 = inv_temperature(a, t) * kLog2e, inv = 1.0 / st.sum;
  const bool rejected = st.c != 0.0;
  load_powers(s_pow);
  __syncthreads();
  const Weigher weigh(s_pow, st.max, it2);
  double2* sums = reinterpret_cast<double2*>(ws + L.off_sum) + (size_t)t * L.splits;
  if (split < L.splits) {
    float x[kPer], q[kPer] = {};
    logits16(a, st.row, split * kChunk + lane * kPer, x);
    if (rejected) draft16(a, st.row, split * kChunk + lane * kPer, q);
    double r = 0.0, p = 0.0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const double w = weigh(x[i]) * inv;
      p += w;
      r += fmax(w - st.c * (double)q[i], 0.0);
    }
    r = wave_sum(r);
    p = wave_sum(p);
    if (lane == 0) {
      __hip_atomic_store(&sums[split].x, r, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __hip_atomic_store(&sums[split].y, p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  // hand-off without a device-scope fence (it would write back the whole L2):
  // the sums went through to the coherent level; wait for them, then count
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0);
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __syncthreads();
  if (tid == 0) s_last = atomicAdd(reinterpret_cast<uint32_t*>(ws + L.off_cnt) + t, 1u) == gridDim.x - 1 ? 1 : 0;
  __syncthreads();
  if (!s_last) return;

  bool residual = true;
  auto sum_of = [&](int i) {
    return __hip_atomic_load(residual ? &sums[i].x : &sums[i].y, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  };
  double total = 0.0;
  for (int i = tid; i < L.splits; i += kThreads) total += sum_of(i);
  total = block_sum<kThreads>(total, s_red);
  if (!(total > 0.0)) {
    residual = false;
    total = 0.0;
    for (int i = tid; i < L.splits; i += kThreads) total += sum_of(i);
    total = block_sum<kThreads>(total, s_red);
  }
  const Found f = find_chunk<kThreads>(sum_of, L.splits, (double)a.u_bonus[t] * total, s_red, s_search);
  constexpr int N = kChunk / kThreads;
  double w[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int tok = f.chunk * kChunk + tid * N + i;
    w[i] = 0.0;
    if (tok < a.vocab) {
      w[i] = weigh(logit(a, st.row, tok)) * inv;
      if (residual && rejected) w[i] = fmax(w[i] - st.c * (double)a.draft[(size_t)st.row * a.vocab + tok], 0.0);
    }
  }
  const int pick = find_token<kThreads>(w, f.rest, s_red, s_search);
  if (tid == 0) a.bonus[t] = f.chunk * kChunk + pick;
}

}  // namespace

size_t tree_sampled_ws_bytes(int num_trees, int total, int vocab) { return layout_of(num_trees, total, vocab).total; }

hipError_t launch_tree_sampled(const SampledArgs& a, hipStream_t s) {
  const int groups = ((a.vocab + kChunk - 1) / kChunk + kWaves - 1) / kWaves;
  // one chunk a wave until the waves fill the card (8192 of them), then up to 8
  // (512 rows of 152064: 85 us, 89 with one each; 9 rows: 24 us, 31 with 8 each)
  const int64_t waves = (int64_t)groups * kWaves * a.total;
  const int each = (int)(waves <= 8192 ? 1 : waves >= 8 * 8192 ? 8 : (waves + 8191) / 8192);
  hipLaunchKernelGGL(sampled_stat_kernel, dim3((groups + each - 1) / each, a.total), dim3(kThreads), 0, s, a, each);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.draft)
    hipLaunchKernelGGL(sampled_walk_kernel<1024>, dim3(a.num_trees), dim3(1024), 0, s, a);
  else
    hipLaunchKernelGGL(sampled_walk_kernel<256>, dim3(a.num_trees), dim3(256), 0, s, a);
  e = hipGetLastError();
  if (e != hipSuccess || !a.draft) return e;
  hipLaunchKernelGGL(sampled_draw_kernel, dim3(groups, a.num_trees), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace w12
