// KV cache of the verify pass (gfx950): appending a step's rows with the
// position rotation, and committing the accepted ones.
//
// Greedy verification ("SpecPilot ..." summary, section 4.3) runs the target
// over a tree of drafted rows and keeps one root path. The cache therefore
// holds two kinds of rows: committed tokens in whole blocks ("pages") of
// 8-bit codes with one scale for each block, head and K or V; and "recent"
// rows in bf16: the committed tokens of the last, unfinished block, then the
// step's drafted rows. A block is quantised once, when its last token is
// committed, from the bf16 rows: the codes depend on the accepted tokens
// alone, never on rejected drafts or on how tokens were grouped into steps.
#include "kv_internal.h"
#include "w12_device.h"

namespace w12 {
namespace {

__device__ __forceinline__ float bf16_f32(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// ---------------------------------------------------------------------------- append

constexpr int kAppendThreads = 256;

__device__ __forceinline__ void load8(const void* p, int f32, size_t at, float (&x)[8]) {
  if (f32) {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    const float4 a = f[0], b = f[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}
__device__ __forceinline__ float load1(const void* p, int f32, size_t at) {
  return f32 ? static_cast<const float*>(p)[at] : bf16_f32(static_cast<const uint16_t*>(p)[at]);
}

// One workgroup per row and 2048 of its values; a thread takes 8 neighbouring
// dims of one head. Rotation in fp32, each product and sum rounded by itself
// (no contraction), one rounding to bf16 at the end. Bound by latency: a row's
// sequence, its parents and its position are found first, a chain of loads, so
// one row takes 5 us, 192 rows 8 (5 MB), 512 fp32 rows of 8192 15 (25 MB, 1.7 TB/s;
// values go out two bytes at a time, as their order has tokens innermost).
__global__ __launch_bounds__(kAppendThreads) void kv_append_kernel(AppendArgs a) {
  __shared__ int s_parent[kStepRows];
  __shared__ int s_seq, s_bad;
  const int tid = threadIdx.x, row = blockIdx.x;
  if (tid == 0) {
    s_seq = a.st.num_seq;
    s_bad = 0;
  }
  __syncthreads();
  for (int s = tid; s < a.st.num_seq; s += kAppendThreads)
    if (rows_meet(a.st.row_off, a.st.total, s, row, 1)) atomicMin(&s_seq, s);
  __syncthreads();
  const int s = s_seq;
  if (s >= a.st.num_seq) return;  // a row of no sequence stays as it is
  const SeqView v = seq_view(a.c, a.st, s);
  int bad = v.ok ? 0 : 1, none = 0;
  const int r = row - v.row0;
  for (int j = tid; j < s; j += kAppendThreads) {
    if (rows_meet(a.st.row_off, a.st.total, j, v.row0, v.rows)) none = 1;
    if (a.st.slot && a.st.slot[j] == v.slot) bad = 1;  // a slot of an earlier sequence would be written twice
  }
  int depth = r;
  if (a.st.parent && v.ok) {
    for (int i = tid; i < v.rows; i += kAppendThreads) {
      const int p = a.st.parent[v.row0 + i];
      s_parent[i] = p;
      if (i == 0 ? p != -1 : (p < 0 || p >= i)) bad = 1;
    }
  }
  if (bad) atomicOr(&s_bad, 1);
  if (none) atomicOr(&s_bad, 2);
  __syncthreads();
  bad = s_bad;
  if (bad & 2) return;
  if (a.st.parent && !bad) {
    depth = 0;
    for (int i = r; i > 0; i = s_parent[i]) ++depth;
  }
  const int pos = v.len + depth;
  const int dim = a.c.dim, heads = a.q_heads + 2 * a.c.kv_heads;
  const int at = blockIdx.y * (kAppendThreads * 8) + tid * 8;
  if (at >= heads * dim) return;
  const int head = at / dim, d0 = at - head * dim;
  const size_t base = (size_t)row * heads * dim;
  uint16_t* qdst = a.q + (size_t)row * a.q_heads * dim + at;
  if (bad || pos >= a.positions) {  // reported through the outputs: NaN
    const uint4 nan = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
    if (head < a.q_heads) *reinterpret_cast<uint4*>(qdst) = nan;
    if (bad || head < a.q_heads) return;
  }
  float x[8], y[8];
  load8(a.qkv, a.qkv_f32, base + at, x);
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = x[i];
  if (head < a.q_heads + a.c.kv_heads && d0 < a.rot) {
#pragma clang fp contract(off)
    if (pos < a.positions) {
      const float* cs = a.rope + (size_t)pos * a.rot;
      const int half = a.rot >> 1;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int d = d0 + i;
        if (d < a.rot) {
          if (a.interleaved) {
            const float c = cs[d >> 1], sn = cs[half + (d >> 1)];
            const float o = x[i ^ 1];
            y[i] = (d & 1) ? x[i] * c + o * sn : x[i] * c - o * sn;
          } else {
            const int f = d < half ? d : d - half;
            const float c = cs[f], sn = cs[half + f];
            const float o = load1(a.qkv, a.qkv_f32, base + (size_t)head * dim + (d < half ? d + half : d - half));
            y[i] = d < half ? x[i] * c - o * sn : x[i] * c + o * sn;
          }
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = __builtin_nanf("");
    }
  }
  uint16_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = f32_to_bf16_rne(y[i]);
  const uint4 o = make_uint4(b[0] | ((uint32_t)b[1] << 16), b[2] | ((uint32_t)b[3] << 16),
                             b[4] | ((uint32_t)b[5] << 16), b[6] | ((uint32_t)b[7] << 16));
  if (head < a.q_heads) {
    *reinterpret_cast<uint4*>(qdst) = o;
  } else if (head < a.q_heads + a.c.kv_heads) {
    uint16_t* k = a.c.recent + recent_at(a.c, a.layer, v.slot, head - a.q_heads, 0);
    *reinterpret_cast<uint4*>(k + key_at(v.tail + r, d0, dim)) = o;
  } else {
    uint16_t* w = a.c.recent + recent_at(a.c, a.layer, v.slot, head - a.q_heads - a.c.kv_heads, 1);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[value_at(v.tail + r, d0 + i, dim)] = b[i];
  }
}

// ---------------------------------------------------------------------------- commit

constexpr int kCommitThreads = 256;
// A block's least scale, as a power of two: the attention multiplies its
// probabilities by the scale, and they must not fall out of fp32's range.
constexpr int kLeastScale = -90;

// What a sequence commits, the same in every workgroup: n accepted rows and
// the recent place each comes from. Invalid where the path is no ascending
// run of the sequence's rows from its root, or a page it closes is none.
struct CommitView {
  SeqView v;
  int n;  // accepted rows, root included
  bool ok;
  bool again;  // an earlier sequence names its slot, and speaks for it
};
__device__ __forceinline__ CommitView commit_view(const CommitArgs& a, int s, int* s_src, int* s_bad) {
  const int tid = threadIdx.x;
  if (tid == 0) *s_bad = 0;
  __syncthreads();
  CommitView w;
  w.v = seq_view(a.c, a.st, s);
  const int acc = a.accept_len[s];
  w.n = w.v.ok ? acc + 1 : 0;
  int bad = (!w.v.ok || acc < -1 || acc >= w.v.rows) ? 1 : 0;
  for (int j = tid; j < s; j += blockDim.x) {
    if (a.st.slot && a.st.slot[j] == w.v.slot) bad |= 2;
    if (rows_meet(a.st.row_off, a.st.total, j, w.v.row0, w.v.rows)) bad |= 1;
  }
  if (!bad) {
    for (int j = tid; j < w.n; j += blockDim.x) {
      int p = j;
      if (a.path) {
        p = a.path[w.v.row0 + j];
        if (j == 0 ? p != 0 : (p <= a.path[w.v.row0 + j - 1] || p >= w.v.rows)) bad = 1;
      }
      s_src[j] = w.v.tail + p;
    }
    const int closed = (w.v.tail + w.n) / a.c.page;
    if (w.v.len + w.n > a.c.max_pages * (long long)a.c.page) {
      bad = 1;  // an unfinished block needs its page too: no call takes a length past the page table
    } else {
      for (int b = tid; b < closed; b += blockDim.x) {
        const int id = a.c.table[(size_t)w.v.slot * a.c.max_pages + w.v.full + b];
        if (id < 0 || id >= a.c.num_pages) bad = 1;
      }
    }
  }
  if (bad) atomicOr(s_bad, bad);
  __syncthreads();
  w.ok = *s_bad == 0;
  w.again = *s_bad & 2;
  return w;
}

// 16 values of chunk `ch` of a block of rows whose sources `src(i)` gives:
// keys are 16 dims of one row, values one dim of 16 rows.
template <typename Src>
__device__ __forceinline__ void gather16(const uint16_t* __restrict__ base, int v, int dim, int ch, bool straight, Src src,
                                         uint32_t (&w)[8]) {
  if (straight) {  // rows as they lie: the block has the recent rows' order
    const uint4* p = reinterpret_cast<const uint4*>(base + (size_t)ch * 16);
    const uint4 x = p[0], y = p[1];
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    w[4] = y.x; w[5] = y.y; w[6] = y.z; w[7] = y.w;
    return;
  }
  const int lane = ch & 63, db = (ch >> 6) % (dim >> 5), g = (ch >> 6) / (dim >> 5);
  if (!v) {
    const uint4* p = reinterpret_cast<const uint4*>(base + key_at(src(g * 32 + (lane & 31)), db * 32 + (lane >> 5) * 16, dim));
    const uint4 x = p[0], y = p[1];
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    w[4] = y.x; w[5] = y.y; w[6] = y.z; w[7] = y.w;
  } else {
    const int d = db * 32 + (lane & 31), t0 = g * 32 + (lane >> 5) * 4;
    const int first = src(t0);
    bool run = (first & 31) == (t0 & 31);
#pragma unroll
    for (int i = 0; i < 4; ++i) run = run && src(t0 + 8 * i + 3) == first + 8 * i + 3;
    if (run) {  // strictly ascending sources: equal ends mean 16 rows as they lie
      const uint4* p = reinterpret_cast<const uint4*>(base + value_at(first, d, dim));
      const uint4 x = p[0], y = p[1];
      w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
      w[4] = y.x; w[5] = y.y; w[6] = y.z; w[7] = y.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int t = t0 + (i >> 1) * 8 + (i & 1) * 2;
        w[i] = base[value_at(src(t), d, dim)] | ((uint32_t)base[value_at(src(t + 1), d, dim)] << 16);
      }
    }
  }
}

// One workgroup per layer, kv head, K or V, and sequence. It closes the
// sequence's full blocks one after another, then moves what is left to the
// front; every dest row lies at or before its source and sources ascend, so
// moving in order, reads before writes within a round, never overwrites a
// row that is still to be read. A block stays in registers between its
// maximum and its codes: kPer pieces of 16 values a thread, as few as hold it
// (with 8 for every block: 64 -> 121 us below, 14 -> 20 for the tree). The next
// block's loads are under way meanwhile. 64 layers of 8 heads of 128, 512 prompt
// rows, 8 blocks each: 61 us for 225 MB (3.7 TB/s), bound by the chain load,
// maximum, barrier, codes of a workgroup's blocks; a 32-row tree that closes one
// block (4 heads of 256): 12 us.
template <int kPer>
__global__ __launch_bounds__(kCommitThreads) void kv_commit_kernel(CommitArgs a) {
  __shared__ int s_src[kStepRows];
  __shared__ int s_bad;
  __shared__ uint32_t s_amax[2][kCommitThreads / 64];  // by the block's parity: one barrier a block
  const int tid = threadIdx.x, s = blockIdx.y;
  const int v = blockIdx.x & 1, head = (blockIdx.x >> 1) % a.c.kv_heads, layer = (blockIdx.x >> 1) / a.c.kv_heads;
  const CommitView w = commit_view(a, s, s_src, &s_bad);
  if (!w.ok || w.n == 0) return;
  const int dim = a.c.dim, page = a.c.page, tail = w.v.tail, n = tail + w.n;
  const int closed = n / page, left = n - closed * page;
  uint16_t* base = a.c.recent + recent_at(a.c, layer, w.v.slot, head, v);
  const int chunks = page * dim / 16;
  uint32_t x[kPer][8], next[kPer][8];
  auto fetch = [&](int b, uint32_t (&to)[kPer][8]) __attribute__((always_inline)) {
    auto src = [&](int i) {
      const int r = b * page + i;
      return r < tail ? r : s_src[r - tail];
    };
    const bool straight = !a.path;
    const uint16_t* from = straight ? base + (size_t)b * page * dim : base;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int ch = k * kCommitThreads + tid;
      if (ch < chunks) gather16(from, v, dim, ch, straight, src, to[k]);
    }
  };
  if (closed > 0) fetch(0, x);
  for (int b = 0; b < closed; ++b) {
    if (b + 1 < closed) fetch(b + 1, next);  // in flight while this block is quantised
    uint32_t most = 0;  // largest magnitude's bits: ordered as integers, NaN above infinity
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int ch = k * kCommitThreads + tid;
      if (ch < chunks) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          most = max(most, (x[k][i] << 16) & 0x7FFF0000u);
          most = max(most, x[k][i] & 0x7FFF0000u);
        }
      }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) most = max(most, (uint32_t)__shfl_xor((int)most, o, 64));
    if ((tid & 63) == 0) s_amax[b & 1][tid >> 6] = most;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kCommitThreads / 64; ++i) most = max(most, s_amax[b & 1][i]);
    const float amax = __uint_as_float(most);
    // e4m3: the power of two that brings amax to 448 = 1.75 * 2^8 or below
    // (exact to divide by); int8: amax / 127. A block that holds an infinity
    // or NaN gets a NaN scale: every value of it reads as NaN.
    float scale = 1.0f;
    if (most >= 0x7F800000u) {
      scale = __builtin_nanf("");
    } else if (most != 0) {
      if (a.c.kind == 0) {
        int e;
        const float f = frexpf(amax, &e);
        scale = ldexpf(1.0f, max(e - 9 + (f > 0.875f ? 1 : 0), kLeastScale));
      } else {
        scale = fmaxf(__fdiv_rn(amax, 127.0f), ldexpf(1.0f, kLeastScale));
      }
    }
    const int id = a.c.table[(size_t)w.v.slot * a.c.max_pages + w.v.full + b];
    if (tid == 0) a.c.scales[scale_at(a.c, layer, id, head, v)] = scale;
    // dividing by a power of two is multiplying by its inverse
    const float div = most >= 0x7F800000u ? 1.0f : scale, inv = a.c.kind == 0 ? 1.0f / div : 0.0f;
    uint8_t* dst = a.c.pages + page_at(a.c, layer, id, head, v);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int ch = k * kCommitThreads + tid;
      if (ch < chunks) {
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t p = x[k][2 * j], q = x[k][2 * j + 1];
          const float f0 = __uint_as_float(p << 16), f1 = __uint_as_float(p & 0xFFFF0000u);
          const float f2 = __uint_as_float(q << 16), f3 = __uint_as_float(q & 0xFFFF0000u);
          if (a.c.kind == 0) {
            int c = __builtin_amdgcn_cvt_pk_fp8_f32(f0 * inv, f1 * inv, 0, false);
            o[j] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f2 * inv, f3 * inv, c, true);
          } else {
            auto code = [div](float f) {
              return (uint32_t)(int)fminf(fmaxf(rintf(__fdiv_rn(f, div)), -127.0f), 127.0f) & 0xFFu;
            };
            o[j] = code(f0) | code(f1) << 8 | code(f2) << 16 | code(f3) << 24;
          }
        }
        *reinterpret_cast<uint4*>(dst + (size_t)ch * 16) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[k][i] = next[k][i];
  }
  // rows that stay recent: logical row closed * page + i to place i, where
  // it does not lie there already
  const int first = closed ? 0 : tail;  // without a closed block the tail stays
  __syncthreads();
  // a round moves 8 dims a thread of kTurns times `per` rows (one turn at a time: 66 us, 64 so)
  constexpr int kTurns = 4;
  const int cols = dim / 8, per = kCommitThreads / cols, d0 = tid % cols * 8;
  for (int i0 = first; i0 < left; i0 += kTurns * per) {
    uint16_t t[kTurns][8];
    int from[kTurns];
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
      const int i = i0 + k * per + tid / cols;
      from[k] = i;
      if (i < left) {
        const int r = closed * page + i;
        from[k] = r < tail ? r : s_src[r - tail];
#pragma unroll
        for (int j = 0; j < 8; ++j) t[k][j] = base[v ? value_at(from[k], d0 + j, dim) : key_at(from[k], d0 + j, dim)];
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
      const int i = i0 + k * per + tid / cols;
      if (from[k] != i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) base[v ? value_at(i, d0 + j, dim) : key_at(i, d0 + j, dim)] = t[k][j];
      }
    }
    __syncthreads();
  }
}

// The new lengths, behind the rows in the stream (len_out may be the cache's own).
__global__ __launch_bounds__(64) void kv_commit_len_kernel(CommitArgs a) {
  __shared__ int s_src[kStepRows];
  __shared__ int s_bad;
  const int s = blockIdx.x;
  const CommitView w = commit_view(a, s, s_src, &s_bad);
  const int slot = a.st.slot ? a.st.slot[s] : s;
  if (threadIdx.x != 0 || slot < 0 || slot >= a.c.slots || w.again) return;
  a.len_out[slot] = w.ok ? w.v.len + w.n : -1;
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs& a, hipStream_t s) {
  const int width = (a.q_heads + 2 * a.c.kv_heads) * a.c.dim;
  const dim3 grid(a.st.total, (width + kAppendThreads * 8 - 1) / (kAppendThreads * 8));
  hipLaunchKernelGGL(kv_append_kernel, grid, dim3(kAppendThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_kv_commit(const CommitArgs& a, hipStream_t s) {
  const dim3 grid(a.c.layers * a.c.kv_heads * 2, a.st.num_seq), block(kCommitThreads);
  const int pieces = (a.c.page * a.c.dim + kCommitThreads * 16 - 1) / (kCommitThreads * 16);  // 1 .. 8
  if (pieces <= 1)
    hipLaunchKernelGGL(kv_commit_kernel<1>, grid, block, 0, s, a);
  else if (pieces <= 2)
    hipLaunchKernelGGL(kv_commit_kernel<2>, grid, block, 0, s, a);
  else if (pieces <= 4)
    hipLaunchKernelGGL(kv_commit_kernel<4>, grid, block, 0, s, a);
  else
    hipLaunchKernelGGL(kv_commit_kernel<8>, grid, block, 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kv_commit_len_kernel, dim3(a.st.num_seq), dim3(64), 0, s, a);
  return hipGetLastError();
}

}  // namespace w12
