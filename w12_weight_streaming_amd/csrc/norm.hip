// Norms, gates and residuals between two products (gfx950).
//
// t = y, normed, gated; h += scale t; out = norm of h (or t). Every tensor is
// read and written once: a row stays in registers between its sums of squares
// and its outputs, 8 neighbouring values a thread. Groups of up to 256 values
// are 1 to 32 lanes of one wave, so their sums need no barrier; wider ones a
// workgroup, of as many threads as give each 8 values (up to 8192), then 16 or 32.
// Bound by bytes at many rows, else by two loads' and one reduction's latency:
// 32 x 5120 bf16 with a residual 4.3 us; 512 x 5120 fp32 with one 9.9 us for 36.7 MB
// (3.7 TB/s); 192 x 48 heads of 128 with gates 4.6 us. A part of a wave
// against a workgroup, rows x groups: 192 x 48 of 128 4.1 us / 6.5, 512 x 16 of 256 5.0 /
// 6.5, 192 x 48 of 256 5.5 / 6.9, 32 x 1 of 256 3.3 / 3.1, 32 x 1 of 512 3.5 / 3.1, 512 x 8
// of 512 5.0 / 4.7, 192 x 48 of 512 8.6 / 7.6. Widths above 16384 (32 values a thread of
// 1024, at most 128 registers) spill 11 to 16 registers.
#include "delta_internal.h"
#include "w12_device.h"

namespace w12 {
namespace {

constexpr int kNarrow = 256;         // widest group of a part of a wave
constexpr int kNarrowThreads = 256;  // of a workgroup of such groups
constexpr int kMostThreads = 1024;

// 8 values from `at`, of `n` that are there (n >= 8: all). Vec: rows and
// groups begin at multiples of 16 bytes and hold a multiple of 8 values.
template <bool Vec>
__device__ __forceinline__ void load8(const void* p, int f32, size_t at, int n, float (&x)[8]) {
  if (f32) {
    const float* f = static_cast<const float*>(p) + at;
    if constexpr (Vec) {
      const float4 a = reinterpret_cast<const float4*>(f)[0], b = reinterpret_cast<const float4*>(f)[1];
      x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
      x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = i < n ? f[i] : 0.0f;
    }
  } else {
    const uint16_t* h = static_cast<const uint16_t*>(p) + at;
    if constexpr (Vec) {
      const uint4 v = *reinterpret_cast<const uint4*>(h);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = i < n ? bf16_to_f32(h[i]) : 0.0f;
    }
  }
}

// Writes 8 values as bf16 (rounded to nearest even) or fp32; x becomes what was stored.
template <bool Vec>
__device__ __forceinline__ void store8(void* p, int f32, size_t at, int n, float (&x)[8]) {
  if (f32) {
    float* f = static_cast<float*>(p) + at;
    if constexpr (Vec) {
      reinterpret_cast<float4*>(f)[0] = make_float4(x[0], x[1], x[2], x[3]);
      reinterpret_cast<float4*>(f)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) f[i] = x[i];
    }
    return;
  }
  uint16_t* h = static_cast<uint16_t*>(p) + at;
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    b[i] = bf16_pair(x[2 * i], x[2 * i + 1]);
    x[2 * i] = __uint_as_float(b[i] << 16);
    x[2 * i + 1] = __uint_as_float(b[i] & 0xFFFF0000u);
  }
  if constexpr (Vec) {
    *reinterpret_cast<uint4*>(h) = make_uint4(b[0], b[1], b[2], b[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) h[i] = (uint16_t)(b[i >> 1] >> (i & 1) * 16);
  }
}

// 1 / sqrt(sum / width + eps) of a group, its threads' shares summed by `all`.
template <int V, typename All>
__device__ __forceinline__ float inverse_rms(const NormArgs& a, const float (&t)[V][8], All all) {
  float sum = 0.0f;
#pragma unroll
  for (int k = 0; k < V; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += t[k][i] * t[k][i];
  return 1.0f / sqrtf(all(sum) / (float)a.width + a.eps);
}

// One group of one row: the thread holds V pieces of 8 values, from value c, then `step` further.
template <bool Vec, int V, typename All>
__device__ __forceinline__ void norm_group(const NormArgs& a, int64_t row, int group, int c, int step, All all_first, All all_last) {
  const size_t wide = (size_t)a.groups * a.width, col = (size_t)group * a.width;
  const size_t at_y = (size_t)row * a.y_stride + col, at_g = (size_t)row * a.gate_stride + col, at = (size_t)row * wide + col;
  // weights too, unless several pieces a thread would take too many registers
  constexpr bool W = V == 1;
  float t[V][8], h[V][8], z[V][8], p[1][8], w[1][8];
  int n[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {  // all loads first
    const int d = c + k * step;
    n[k] = a.width - d;
    if (n[k] > 0) {
      if (a.y) load8<Vec>(a.y, a.y_f32, at_y + d, n[k], t[k]);
      if (a.h) load8<Vec>(a.h, a.h_f32, at + d, n[k], h[k]);
      if (a.gate) load8<Vec>(a.gate, a.gate_f32, at_g + d, n[k], z[k]);
      if (W && a.post_weight) load8<Vec>(a.post_weight, 1, d, n[k], p[0]);
      if (W && a.weight) load8<Vec>(a.weight, 1, d, n[k], w[0]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) t[k][i] = h[k][i] = 0.0f;
    }
  }
  if (a.post_weight) {
    const float f = inverse_rms<V>(a, t, all_first);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if (n[k] <= 0) continue;
      if (!W) load8<Vec>(a.post_weight, 1, c + k * step, n[k], p[0]);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[k][i] *= f * p[0][i];
    }
  }
#pragma unroll
  for (int k = 0; k < V; ++k) {
    if (n[k] <= 0) continue;
    if (a.gate)
#pragma unroll
      for (int i = 0; i < 8; ++i) t[k][i] *= silu(z[k][i]);
    if (a.h) {
      if (a.y) {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[k][i] += a.scale * t[k][i];
        store8<Vec>(a.h, a.h_f32, at + c + k * step, n[k], h[k]);
        if constexpr (!Vec)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i >= n[k]) h[k][i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) t[k][i] = h[k][i];
    }
  }
  if (a.weight) {
    const float f = inverse_rms<V>(a, t, all_last);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if (n[k] <= 0) continue;
      if (!W) load8<Vec>(a.weight, 1, c + k * step, n[k], w[0]);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[k][i] *= f * w[0][i];
    }
  }
#pragma unroll
  for (int k = 0; k < V; ++k)
    if (n[k] > 0) store8<Vec>(a.out, 0, at + c + k * step, n[k], t[k]);
}

// Groups of up to 256 values: `lanes` (a power of two) neighbouring lanes each.
template <bool Vec>
__global__ __launch_bounds__(kNarrowThreads) void norm_narrow_kernel(NormArgs a, int lanes) {
  const int per = kNarrowThreads / lanes, mine = threadIdx.x / lanes, c = (threadIdx.x & (lanes - 1)) * 8;
  const auto all = [&](float x) {
    for (int m = 1; m < lanes; m <<= 1) x += __shfl_xor(x, m);
    return x;
  };
  const int64_t items = a.rows * a.groups;
  for (int64_t first = (int64_t)blockIdx.x * per; first < items; first += (int64_t)gridDim.x * per) {
    const int64_t row0 = first / a.groups;  // the same for all threads
    const uint32_t from = (uint32_t)(first - row0 * a.groups) + mine, up = from / (uint32_t)a.groups;
    if (first + mine < items) norm_group<Vec, 1>(a, row0 + up, (int)(from - up * a.groups), c, 0, all, all);
  }
}

// Wider groups: a workgroup each.
template <bool Vec, int V>
__global__ __launch_bounds__(kMostThreads) void norm_wide_kernel(NormArgs a) {
  __shared__ float part[2][kMostThreads / 64];
  const int waves = blockDim.x >> 6;
  int turn = 0;
  const auto all = [&](float x) {  // the two sums of a row use an array each; between rows there is a barrier
    for (int m = 1; m < 64; m <<= 1) x += __shfl_xor(x, m);
    if ((threadIdx.x & 63) == 0) part[turn][threadIdx.x >> 6] = x;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < waves; ++i) s += part[turn][i];
    turn ^= 1;
    return s;
  };
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    norm_group<Vec, V>(a, row, blockIdx.y, threadIdx.x * 8, blockDim.x * 8, all, all);
    if (row + gridDim.x < a.rows) __syncthreads();
  }
}

bool fits16(const void* p, int f32, int64_t stride) {
  const int64_t size = f32 ? 4 : 2;
  return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * size % 16 == 0);
}

template <bool Vec>
void launch(const NormArgs& a, hipStream_t s) {
  if (a.width <= kNarrow) {
    int lanes = 1;
    while (lanes * 8 < a.width) lanes <<= 1;
    const int64_t per = kNarrowThreads / lanes, blocks = (a.rows * a.groups + per - 1) / per;
    norm_narrow_kernel<Vec><<<(unsigned)(blocks < (1 << 22) ? blocks : 1 << 22), kNarrowThreads, 0, s>>>(a, lanes);
    return;
  }
  const int pieces = (a.width + 7) / 8, v = (pieces + kMostThreads - 1) / kMostThreads;
  const int threads = (v == 1 ? (pieces + 63) / 64 * 64 : kMostThreads);
  const dim3 grid((unsigned)(a.rows < (1 << 20) ? a.rows : 1 << 20), a.groups);
  if (v == 1)
    norm_wide_kernel<Vec, 1><<<grid, threads, 0, s>>>(a);
  else if (v == 2)
    norm_wide_kernel<Vec, 2><<<grid, threads, 0, s>>>(a);
  else
    norm_wide_kernel<Vec, 4><<<grid, threads, 0, s>>>(a);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
  const int64_t wide = (int64_t)a.groups * a.width;
  const bool vec = a.width % 8 == 0 && fits16(a.y, a.y_f32, a.y_stride) && fits16(a.gate, a.gate_f32, a.gate_stride) &&
                   fits16(a.h, a.h_f32, wide) && fits16(a.out, 0, wide) && fits16(a.post_weight, 1, 0) &&
                   fits16(a.weight, 1, 0);
  vec ? launch<true>(a, s) : launch<false>(a, s);
  return hipGetLastError();
}

}  // namespace w12
