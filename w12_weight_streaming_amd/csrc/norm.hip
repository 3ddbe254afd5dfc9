// Norms, gates and residuals between two products (gfx950).
#include "delta_internal.h"
#include "w12_device.h"

namespace w12 {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float load1(const void* p, int f32, size_t at) {
  return f32 ? static_cast<const float*>(p)[at] : bf16_to_f32(static_cast<const uint16_t*>(p)[at]);
}

__device__ __forceinline__ float block_sum(float x) {
  __shared__ float part[kThreads / 64];
  for (int m = 1; m < 64; m <<= 1) x += __shfl_xor(x, m);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
  __syncthreads();
  float s = 0;
  for (int i = 0; i < kThreads / 64; ++i) s += part[i];
  return s;
}

// One workgroup per row and group.
__global__ __launch_bounds__(kThreads) void norm_kernel(NormArgs a) {
  const int64_t row = blockIdx.x;
  const int group = blockIdx.y, tid = threadIdx.x;
  const size_t wide = (size_t)a.groups * a.width, col = (size_t)group * a.width;
  float post = 1.0f, sum = 0.0f;
  if (a.post_weight) {
    for (int i = tid; i < a.width; i += kThreads) {
      const float x = load1(a.y, a.y_f32, row * a.y_stride + col + i);
      sum += x * x;
    }
    post = 1.0f / sqrtf(block_sum(sum) / a.width + a.eps);
  }
  const auto value = [&](int i) {
    const size_t at = row * wide + col + i;
    if (!a.y) return load1(a.h, a.h_f32, at);
    float t = load1(a.y, a.y_f32, row * a.y_stride + col + i);
    if (a.post_weight) t = t * post * a.post_weight[i];
    if (a.gate) {
      const float z = load1(a.gate, a.gate_f32, row * a.gate_stride + col + i);
      t *= z / (1.0f + __expf(-z));
    }
    return t;
  };
  sum = 0.0f;
  for (int i = tid; i < a.width; i += kThreads) {
    float t = value(i);
    const size_t at = row * wide + col + i;
    if (a.h && a.y) {
      t = load1(a.h, a.h_f32, at) + a.scale * t;
      if (a.h_f32) {
        static_cast<float*>(a.h)[at] = t;
      } else {
        const uint16_t b = f32_to_bf16_rne(t);
        static_cast<uint16_t*>(a.h)[at] = b;
        t = bf16_to_f32(b);
      }
    }
    sum += t * t;
  }
  const float f = a.weight ? 1.0f / sqrtf(block_sum(sum) / a.width + a.eps) : 1.0f;
  for (int i = tid; i < a.width; i += kThreads) {
    const size_t at = row * wide + col + i;
    float u = a.h ? load1(a.h, a.h_f32, at) : value(i);
    if (a.weight) u = u * f * a.weight[i];
    a.out[at] = f32_to_bf16_rne(u);
  }
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
  norm_kernel<<<dim3((unsigned)a.rows, a.groups), kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace w12
