// Matrix-core helpers of the recurrent layers (gfx950): states and deltas (fp32)
// times keys and queries (bf16) in three bf16 pieces.
#pragma once

#include <type_traits>

#include "delta_internal.h"
#include "w12_device.h"

namespace w12 {

// The thread's place, derived anew in each phase of a kernel: kept from one
// phase to the next, addresses made of it take more registers than the states.
__device__ __forceinline__ int thread_now() {
  int t = threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
}

typedef float f32x4 __attribute__((ext_vector_type(4)));

// `bytes` behind a uniform address: in this form the address stays in scalar
// registers and the lane's part in one vector register.
template <typename T>
__device__ __forceinline__ T* behind(T* base, uint32_t bytes) {
  using Byte = std::conditional_t<std::is_const_v<T>, const char, char>;
  return reinterpret_cast<T*>(reinterpret_cast<Byte*>(base) + bytes);
}

// Reads and writes of states, which no call comes back to before others have
// gone through the caches: past them, if the lane has two neighbouring dims (a
// wave's 128 bytes a row are whole lines; of 64 bytes the caches join the halves).
typedef float f32x2 __attribute__((ext_vector_type(2)));
template <int NC>
__device__ __forceinline__ void read_dims(const float* p, float (&x)[NC]) {
  if constexpr (NC == 2) {
    const f32x2 y = __builtin_nontemporal_load(reinterpret_cast<const f32x2*>(p));
    x[0] = y[0];
    x[1] = y[1];
  } else {
    x[0] = *p;
  }
}
template <int NC>
__device__ __forceinline__ void write_dims(float* p, const float (&x)[NC]) {
  if constexpr (NC == 2)
    __builtin_nontemporal_store(f32x2{x[0], x[1]}, reinterpret_cast<f32x2*>(p));
  else
    *p = x[0];
}

// The NC * 16 columns of a head's state that a wave holds, from value dim vw,
// NC neighbouring ones a lane, in the layout of the products: a uniform part of
// each address, and the lane's in 32 bits.
template <int VD, int NC>
__device__ __forceinline__ uint32_t state_place(int vw) {
  const int lane = thread_now() & 63;
  return (uint32_t)(4 * (4 * (lane >> 4) * VD + vw + (lane & 15) * NC));  // in bytes
}
template <int KT, int VD, int NC>
__device__ __forceinline__ void load_state(const float* state, int vw, f32x4 (&S)[KT][NC]) {
  const uint32_t at = state_place<VD, NC>(vw);
#pragma unroll
  for (int t = 0; t < KT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float x[NC];
      read_dims<NC>(behind(state + (16 * t + r) * VD, at), x);
#pragma unroll
      for (int c = 0; c < NC; ++c) S[t][c][r] = x[c];
    }
}
template <int KT, int VD, int NC>
__device__ __forceinline__ void store_state(float* state, int vw, const f32x4 (&S)[KT][NC]) {
  const uint32_t at = state_place<VD, NC>(vw);
#pragma unroll
  for (int t = 0; t < KT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float x[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) x[c] = S[t][c][r];
      write_dims<NC>(behind(state + (16 * t + r) * VD, at), x);
    }
}

// Result layout of every product here, lane l of a wave: column l % 16, row
// 4 (l / 16) + r in value r. An operand's depth is taken in the order (l / 16,
// r) too, so a result serves as the next product's operand as it stands.
__device__ __forceinline__ f32x4 mfma_bf16(const uint4& a, const uint4& b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
// 16 deep in fp32.
__device__ __forceinline__ f32x4 mfma_f32(const f32x4& a, const f32x4& b, f32x4 c) {
#pragma unroll
  for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[r], c, 0, 0, 0);
  return c;
}

// 8 fp32 values as three bf16 operands whose sum they are: each piece is the
// value's (then the rest's) top 16 bits, and the rests are exact.
__device__ __forceinline__ void split3(const f32x4& x, const f32x4& y, uint4& hi, uint4& mid, uint4& lo) {
  uint32_t h[4], m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = i < 2 ? x[2 * i] : y[2 * i - 4], b = i < 2 ? x[2 * i + 1] : y[2 * i - 3];
    const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
    h[i] = __builtin_amdgcn_perm(ub, ua, 0x07060302u);
    const float ra = a - __uint_as_float(ua & 0xFFFF0000u), rb = b - __uint_as_float(ub & 0xFFFF0000u);
    const uint32_t va = __float_as_uint(ra), vb = __float_as_uint(rb);
    m[i] = __builtin_amdgcn_perm(vb, va, 0x07060302u);
    const float sa = ra - __uint_as_float(va & 0xFFFF0000u), sb = rb - __uint_as_float(vb & 0xFFFF0000u);
    l[i] = __builtin_amdgcn_perm(__float_as_uint(sb), __float_as_uint(sa), 0x07060302u);
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  mid = make_uint4(m[0], m[1], m[2], m[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// What rows add to a state, S <- keep S + add, rounded once at the state's size:
// the pieces' products are gathered from zero, as each one that went into S by
// itself would round it again.
__device__ __forceinline__ void join_state(f32x4& S, float keep, const f32x4& add) {
#pragma unroll
  for (int r = 0; r < 4; ++r) S[r] = __builtin_fmaf(keep, S[r], add[r]);
}

// 8 bf16 of a row (two 8-byte pieces, 16 values apart): depths 4 (l / 16) + r of two neighbouring tiles of 16.
__device__ __forceinline__ uint4 fragment(const uint16_t* p) {
  const uint2 a = *reinterpret_cast<const uint2*>(p), b = *reinterpret_cast<const uint2*>(p + 16);
  return make_uint4(a.x, a.y, b.x, b.y);
}

// Two rows' 8 values each, as pairs for an array with rows innermost, `stride` values a column.
__device__ __forceinline__ void store_turned(uint16_t* to, int stride, const uint4& a, const uint4& b) {
  const uint32_t u[2][4] = {{a.x, a.y, a.z, a.w}, {b.x, b.y, b.z, b.w}};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<uint32_t*>(to + i * stride) =
        __builtin_amdgcn_perm(u[1][i >> 1], u[0][i >> 1], (i & 1) ? 0x07060302u : 0x05040100u);
}

// Infinities and NaN among bf16 values: their exponent's ones carry into the
// sign's place, and several words' sums can be looked at together.
__device__ __forceinline__ uint32_t odd_sum(uint32_t w) { return (w & 0x7F807F80u) + 0x00800080u; }
__device__ __forceinline__ uint32_t odd_sum(const uint4& x) { return odd_sum(x.x) | odd_sum(x.y) | odd_sum(x.z) | odd_sum(x.w); }
__device__ __forceinline__ bool is_odd(uint32_t sums) { return sums & 0x80008000u; }
__device__ __forceinline__ bool odd32(float x) { return !(fabsf(x) <= 3.4e38f); }

// One tile of x . k, transposed, over KD dims: lane (l / 16, l % 16) holds row l % 16 of x, rows 4 (l / 16) + r
// of k, so that it serves as a product's first operand. x, k: the tile's first rows, `stride` values apart.
template <int KD>
__device__ __forceinline__ f32x4 pair_tile(const uint16_t* x, const uint16_t* k, int stride, int lane) {
  const int at = (lane & 15) * stride + 4 * (lane >> 4);
  f32x4 acc = {0, 0, 0, 0};
#pragma unroll
  for (int t = 0; t < KD / 32; ++t) acc = mfma_bf16(fragment(k + at + 32 * t), fragment(x + at + 32 * t), acc);
  return acc;
}

// (I + L)^-1 of a diagonal tile from -L, a column per lane of the first 16, by
// forward substitution: L's products of keys make it as well conditioned as the
// rule itself, where powers of L would cancel. Wide: all rows of L are read at
// once, into 144 registers, and each value goes into all the sums that wait
// for it (900 cycles); else rows a few at a time, each value's sum at once (2000),
// and tiles of up to eight rows stop there.
template <int First, int Last>
__device__ __forceinline__ void substitute(const f32x4* low, int c, float (&x)[16]) {
#pragma unroll
  for (int i = First; i < Last; ++i) {
    float y = i == c ? 1.0f : 0.0f;
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
  }
  __builtin_amdgcn_sched_barrier(0);
}
template <bool Wide>
__device__ __forceinline__ void invert(const f32x4* low, f32x4* inv, int n) {
  const int lane = thread_now() & 63, c = lane & 15;
  float x[16];
  if constexpr (Wide) {
    f32x4 l[16][4];
#pragma unroll
    for (int i = 1; i < 16; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        if (4 * g < i) l[i][g] = low[g * 16 + i];
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = i == c ? 1.0f : 0.0f;
#pragma unroll
    for (int j = 0; j < 15; ++j)
#pragma unroll
      for (int i = j + 1; i < 16; ++i) x[i] += l[i][j >> 2][j & 3] * x[j];
  } else {
    substitute<0, 8>(low, c, x);
    if (n > 8) {  // the same for all lanes
      substitute<8, 12>(low, c, x);
      substitute<12, 16>(low, c, x);
    } else {
#pragma unroll
      for (int i = 8; i < 16; ++i) x[i] = i == c ? 1.0f : 0.0f;
    }
  }
  if (lane < 16) {
    float* o = reinterpret_cast<float*>(inv);
#pragma unroll
    for (int i = 0; i < 16; ++i) o[((c >> 2) * 16 + i) * 4 + (c & 3)] = x[i];
  }
}

}  // namespace w12
