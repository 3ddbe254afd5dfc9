// Attention of a step's rows over the 8-bit paged cache (gfx950).
//
// Row i of sequence s attends to the sequence's committed tokens and to its
// own ancestors among the step's rows, itself included:
//   out = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - max)
// in one pass over the tokens with the running maximum m and sum l of the
// softmax. The scores come transposed, S^T = K Q^T, so a lane of the 32x32x16
// matrix instruction owns one query row: its m and l are one register each,
// and its 16 probabilities per group of 32 tokens are, in the order in which
// they come out, the B operand of O^T = V^T P^T. Pages hold keys and values in
// the operands' order (kv_internal.h), so nothing is transposed or shuffled:
// a 1 KB wave-wide load is one operand of 8-bit codes, and the conversion to
// bf16 is exact (at most 8 significant bits). The block's scales multiply the
// scores and the probabilities in fp32.
//
// Work split: an item is (sequence, kv head, tile of 32 query rows); its
// units are groups of 32 tokens, pages first, then the recent rows. The units
// of all items in order are cut into equal runs, one for each workgroup, so
// ragged batches balance; within a run the four waves take units in turn. An
// item that several workgroups share is joined by the last of them to arrive,
// in workgroup order: results are bitwise reproducible.
#include "kv_internal.h"
#include "w12_device.h"

namespace w12 {
namespace {

constexpr int kThreads = 256, kWaves = 4;
constexpr int kTile = 32;        // query rows of an item
constexpr int kUnitsPerWg = 4;   // fewest units worth a workgroup of their own
constexpr float kLog2e = 1.44269504088896340736f;
// a new maximum is taken when a score passes the running one by this much
// (in powers of two): until then probabilities may reach 2^8, which neither
// fp32 sums nor bf16 operands lose anything by, and the rescaling is skipped
constexpr float kSlack = 8.0f;
constexpr float kFloor = -3.402823466e38f;  // running maximum before the first score

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;
constexpr int kRawBufferWord3 = 0x00020000;
constexpr int kDeviceScope = 16;  // sc1: coherent across XCDs

__device__ __forceinline__ rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)b);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32));
  void* ub = reinterpret_cast<void*>(((uint64_t)hi << 32) | lo);
  return __builtin_amdgcn_make_buffer_rsrc(ub, (short)0, (int)__builtin_amdgcn_readfirstlane(bytes), kRawBufferWord3);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __bf16 x = (__bf16)a, y = (__bf16)b;
  return (uint32_t)__builtin_bit_cast(uint16_t, x) | ((uint32_t)__builtin_bit_cast(uint16_t, y) << 16);
}
__device__ __forceinline__ bf16x8 as_operand(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(bf16x8, u32x4{a, b, c, d});
}

// Four 8-bit codes as bf16 pairs, exactly.
template <int KIND>
__device__ __forceinline__ void codes4(uint32_t x, uint32_t& lo, uint32_t& hi) {
  if constexpr (KIND == 0) {
    lo = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, 1.0f, false));
    hi = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, 1.0f, true));
  } else {
    const uint32_t f0 = __float_as_uint((float)(int8_t)x), f1 = __float_as_uint((float)(int8_t)(x >> 8));
    const uint32_t f2 = __float_as_uint((float)(int8_t)(x >> 16)), f3 = __float_as_uint((float)(int8_t)(x >> 24));
    lo = __builtin_amdgcn_perm(f1, f0, 0x07060302u);
    hi = __builtin_amdgcn_perm(f3, f2, 0x07060302u);
  }
}
template <int KIND>
__device__ __forceinline__ void codes16(const u32x4 x, bf16x8& a, bf16x8& b) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) codes4<KIND>(x[i], w[2 * i], w[2 * i + 1]);
  a = as_operand(w[0], w[1], w[2], w[3]);
  b = as_operand(w[4], w[5], w[6], w[7]);
}

template <int DIM>
struct Acc {
  f32x16 o[DIM / 32];
  float m, l;
};

// One group of 32 scores per row: x = S * c (masked where `see` has no bit),
// then the probabilities, and their operands scaled by `vs`.
template <int DIM>
__device__ __forceinline__ void softmax_step(Acc<DIM>& acc, const f32x16& sc, float c, float vs, uint32_t see, int half,
                                             float (&p)[16], bf16x8 (&pb)[2]) {
  float x[16], mx = kFloor;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    x[r] = sc[r] * c;
    if (!((see >> ((r >> 2) * 8 + half * 4 + (r & 3))) & 1)) x[r] = -__builtin_huge_valf();
    mx = fmaxf(mx, x[r]);
  }
  mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
  if (__any(mx > acc.m + kSlack)) {
    const float nm = fmaxf(acc.m, mx);
    const float al = __builtin_amdgcn_exp2f(acc.m - nm);
    acc.m = nm;
    acc.l *= al;
#pragma unroll
    for (int i = 0; i < DIM / 32; ++i) acc.o[i] *= al;
  }
  float sum = 0.f;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    p[r] = __builtin_amdgcn_exp2f(x[r] - acc.m);
    sum += p[r];
  }
  acc.l += sum;
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack_bf16(p[2 * i] * vs, p[2 * i + 1] * vs);
  pb[0] = as_operand(w[0], w[1], w[2], w[3]);
  pb[1] = as_operand(w[4], w[5], w[6], w[7]);
}

__device__ __forceinline__ int owner_of(int64_t u, int64_t total, int wgs) {
  // the workgroup w with w * total / wgs <= u < (w + 1) * total / wgs
  int w = (int)(((u + 1) * wgs - 1) / total);
  return w;
}

template <int DIM, int KIND>
__global__ __launch_bounds__(kThreads, DIM == 256 ? 1 : 2) void kv_attention_kernel(AttentionArgs a) {
  constexpr int NB = DIM / 32;
  __shared__ int64_t s_first[kStepRows + 1];  // units before each sequence
  __shared__ int64_t s_scan[kThreads];
  __shared__ int s_parent[kStepRows];
  __shared__ uint32_t s_anc[kTile][kStepRows / 32];
  __shared__ float s_ml[kWaves][kTile][2];
  __shared__ int s_bad, s_last;
  __shared__ float s_o[2][kTile * DIM];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 31, half = lane >> 5;
  const int group = a.q_heads / a.c.kv_heads;

  // units of every sequence, then their running sum
  auto tiles_of = [&](const SeqView& v) { return (v.rows * group + kTile - 1) / kTile; };
  auto units_of = [&](const SeqView& v) {
    return v.ok ? v.full * (a.c.page / kGroup) + (v.tail + v.rows + kGroup - 1) / kGroup : 1;
  };
  int64_t mine[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int s = tid * 2 + i;
    mine[i] = 0;
    if (s < a.st.num_seq) {
      const SeqView v = seq_view(a.c, a.st, s);
      mine[i] = (int64_t)tiles_of(v) * a.c.kv_heads * units_of(v);
    }
  }
  s_scan[tid] = mine[0] + mine[1];
  __syncthreads();
  for (int o = 1; o < kThreads; o <<= 1) {
    const int64_t x = tid >= o ? s_scan[tid - o] : 0;
    __syncthreads();
    s_scan[tid] += x;
    __syncthreads();
  }
  {
    const int64_t before = s_scan[tid] - mine[0] - mine[1];
    s_first[tid * 2] = before;
    s_first[tid * 2 + 1] = before + mine[0];
    if (tid == kThreads - 1) s_first[kStepRows] = s_scan[tid];
  }
  __syncthreads();
  const int64_t total = s_first[kStepRows];
  if (total == 0) return;
  const int wgs = (int)min((int64_t)a.G, (total + kUnitsPerWg - 1) / kUnitsPerWg);
  const int wg = blockIdx.x;
  if (wg >= wgs) return;
  const int64_t begin = total * wg / wgs, end = total * (wg + 1) / wgs;

  int seq;  // the first sequence whose units reach past `begin`
  {
    int lo = 0, hi = a.st.num_seq - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (s_first[mid + 1] > begin) hi = mid; else lo = mid + 1;
    }
    seq = lo;
  }

  for (int64_t at = begin; at < end;) {
    while (s_first[seq + 1] <= at) ++seq;
    const SeqView v = seq_view(a.c, a.st, seq);
    const int tiles = tiles_of(v), units = units_of(v);
    const int item = (int)((at - s_first[seq]) / units);
    const int64_t item0 = s_first[seq] + (int64_t)item * units;  // the item's first unit
    const int u0 = (int)(at - item0), u1 = (int)min((int64_t)units, end - item0);
    const int kvh = item / tiles, tile = item % tiles;
    const int first_row = tile * kTile, q_rows = v.rows * group;
    const int my = first_row + col;  // the lane's query row: row my / group, head my % group
    const bool on = my < q_rows && v.ok;
    const int page_units = v.ok ? v.full * (a.c.page / kGroup) : 0;
    bool poison = !v.ok;

    // ancestors of the tile's rows
    const int row_lo = first_row / group, row_hi = min(v.rows, (first_row + kTile - 1) / group + 1);
    __syncthreads();
    if (tid == 0) s_bad = 0;
    __syncthreads();
    if (v.ok && u1 > page_units) {
      if (a.st.parent) {
        int bad = 0;
        for (int i = tid; i < v.rows; i += kThreads) {
          const int p = a.st.parent[v.row0 + i];
          s_parent[i] = p;
          if (i == 0 ? p != -1 : (p < 0 || p >= i)) bad = 1;
        }
        for (int i = tid; i < kTile * (kStepRows / 32); i += kThreads) (&s_anc[0][0])[i] = 0;
        if (bad) s_bad = 1;
        __syncthreads();
        if (!s_bad && row_lo + tid < row_hi) {
          for (int i = row_lo + tid; i >= 0; i = s_parent[i]) s_anc[tid][i >> 5] |= 1u << (i & 31);
        }
      } else {
        for (int i = tid; i < (row_hi - row_lo) * (kStepRows / 32); i += kThreads) {
          const int r = row_lo + i / (kStepRows / 32) - (i % (kStepRows / 32)) * 32;  // highest visible bit
          s_anc[i / (kStepRows / 32)][i % (kStepRows / 32)] = r < 0 ? 0u : r >= 31 ? ~0u : (2u << r) - 1u;
        }
      }
    }
    __syncthreads();
    poison = poison || s_bad;

    // the lane's query row as B operands: dims 32 i + 16 half + 0..15
    bf16x8 qf[NB][2];
    {
      const int r = on ? my / group : 0, h = kvh * group + (on ? my % group : 0);
      const u32x4* p = reinterpret_cast<const u32x4*>(a.q + ((size_t)(v.row0 + r) * a.q_heads + h) * DIM + half * 16);
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        u32x4 x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
        if (on) {
          x = p[i * 4];
          y = p[i * 4 + 1];
        }
        qf[i][0] = __builtin_bit_cast(bf16x8, x);
        qf[i][1] = __builtin_bit_cast(bf16x8, y);
      }
    }
    Acc<DIM> acc;
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc.o[i][r] = 0.f;
    acc.m = kFloor;
    acc.l = 0.f;
    const float c2 = a.scale * kLog2e;

    // pages: units u0 + wave + 4 k below `page_units`, ids and scales of 64 at a time
    const int pu1 = min(u1, page_units);
    const int np = u0 + wave < pu1 ? (pu1 - u0 - wave + kWaves - 1) / kWaves : 0;
    const int per_page = a.c.page / kGroup;
    for (int kb = 0; kb < np; kb += 64) {
      int id = 0;
      float ks = 0.f, vs = 0.f;
      if (kb + lane < np) {
        const int j = (u0 + wave + kWaves * (kb + lane)) / per_page;
        id = a.c.table[(size_t)v.slot * a.c.max_pages + j];
        const bool good = id >= 0 && id < a.c.num_pages;
        if (!good) id = 0;
        const float2 sc = *reinterpret_cast<const float2*>(a.c.scales + scale_at(a.c, a.layer, id, kvh, 0));
        ks = good ? sc.x : __builtin_nanf("");
        vs = sc.y;
      }
      const int cnt = min(64, np - kb);
      u32x4 kr[NB], vr[NB];
      auto load = [&](int k) {
        const int u = u0 + wave + kWaves * (kb + k);
        const int pid = __builtin_amdgcn_readlane(id, k);
        const uint8_t* p = a.c.pages + page_at(a.c, a.layer, pid, kvh, 0) + (size_t)(u % per_page) * (kGroup * DIM) + lane * 16;
        const size_t to_v = (size_t)a.c.page * DIM;
#pragma unroll
        for (int i = 0; i < NB; ++i) kr[i] = *reinterpret_cast<const u32x4*>(p + i * 1024);
#pragma unroll
        for (int i = 0; i < NB; ++i) vr[i] = *reinterpret_cast<const u32x4*>(p + to_v + i * 1024);
      };
      load(0);
      for (int k = 0; k < cnt; ++k) {
        f32x16 sc;
#pragma unroll
        for (int r = 0; r < 16; ++r) sc[r] = 0.f;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          bf16x8 x, y;
          codes16<KIND>(kr[i], x, y);
          sc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, qf[i][0], sc, 0, 0, 0);
          sc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(y, qf[i][1], sc, 0, 0, 0);
        }
        const float ksk = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ks), k));
        const float vsk = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(vs), k));
        u32x4 vn[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i) vn[i] = vr[i];
        if (k + 1 < cnt) load(k + 1);
        float p[16];
        bf16x8 pb[2];
        softmax_step(acc, sc, c2 * ksk, vsk, ~0u, half, p, pb);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          bf16x8 x, y;
          codes16<KIND>(vn[i], x, y);
          acc.o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, pb[0], acc.o[i], 0, 0, 0);
          acc.o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(y, pb[1], acc.o[i], 0, 0, 0);
        }
      }
    }

    // recent rows: the committed tail, then the step's rows
    if (!poison) {
      const uint16_t* kb = a.c.recent + recent_at(a.c, a.layer, v.slot, kvh, 0);
      const uint16_t* vb = a.c.recent + recent_at(a.c, a.layer, v.slot, kvh, 1);
      const int rows = v.tail + v.rows;
      int u = u0 + wave;
      if (u < page_units) u += (page_units - u + kWaves - 1) / kWaves * kWaves;
      for (; u < u1; u += kWaves) {
        const int t0 = (u - page_units) * kGroup;
        const int held = rows - t0 >= 32 ? 32 : rows - t0;  // rows of this group that there are
        const uint32_t there = held == 32 ? ~0u : (1u << held) - 1u;
        f32x16 sc;
#pragma unroll
        for (int r = 0; r < 16; ++r) sc[r] = 0.f;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const u32x4* p = reinterpret_cast<const u32x4*>(kb + (size_t)t0 * DIM + i * 1024 + lane * 16);
          sc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, p[0]), qf[i][0], sc, 0, 0, 0);
          sc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, p[1]), qf[i][1], sc, 0, 0, 0);
        }
        // bit t: the lane's row sees place t0 + t: every tail token, and its ancestors
        uint32_t see = 0;
        if (on) {
          const int rr = my / group - row_lo;
          const int shift = t0 - v.tail;  // the step's row at place t0
          uint32_t w = 0;
          if (shift >= 0) {
            const int k = shift >> 5, b = shift & 31;
            const uint64_t two = (uint64_t)s_anc[rr][k] | ((uint64_t)(k + 1 < kStepRows / 32 ? s_anc[rr][k + 1] : 0u) << 32);
            w = (uint32_t)(two >> b);
          } else if (shift > -32) {
            w = (s_anc[rr][0] << -shift) | ((1u << -shift) - 1u);
          } else {
            w = ~0u;
          }
          see = w & there;
        }
        float p[16];
        bf16x8 pb[2];
        softmax_step(acc, sc, c2, 1.0f, see, half, p, pb);
        // values: a row that is not there, or an infinity or NaN that some
        // query row does not see, must not meet its probability of zero
        u32x4 vr[NB][2];
        uint32_t odd = 0;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const u32x4* q = reinterpret_cast<const u32x4*>(vb + (size_t)t0 * DIM + i * 1024 + lane * 16);
          vr[i][0] = q[0];
          vr[i][1] = q[1];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            // slots 2 e, 2 e + 1: tokens 8 (e >> 1) + 4 half + 2 (e & 1) and the next
            const int t = (e >> 1) * 8 + half * 4 + (e & 1) * 2;
            uint32_t w = vr[i][e >> 2][e & 3];
            w &= ((there >> t) & 1 ? 0xFFFFu : 0u) | ((there >> (t + 1)) & 1 ? 0xFFFF0000u : 0u);
            odd |= (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
            vr[i][e >> 2][e & 3] = w;
          }
        }
        const bool strange = __any(odd);
        if (strange) {
#pragma unroll
          for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              uint32_t w = vr[i][e >> 2][e & 3];
              if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
              if ((w & 0x7F800000u) == 0x7F800000u) w &= 0xFFFFu;
              vr[i][e >> 2][e & 3] = w;
            }
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          acc.o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, vr[i][0]), pb[0], acc.o[i], 0, 0, 0);
          acc.o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, vr[i][1]), pb[1], acc.o[i], 0, 0, 0);
        }
        if (strange) {  // those values again, by themselves, for the rows that see them
          float* sp = &s_o[0][0] + wave * (32 * kTile);  // free until the waves join
#pragma unroll
          for (int r = 0; r < 16; ++r) sp[((r >> 2) * 8 + half * 4 + (r & 3)) * kTile + col] = p[r];
          wave_lds_sync();
          for (int t = 0; t < held; ++t) {
            if (!((see >> t) & 1)) continue;
            const float pt = sp[t * kTile + col];
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
              for (int r = 0; r < 16; ++r) {
                const uint16_t w = vb[value_at(t0 + t, i * 32 + (r >> 2) * 8 + half * 4 + (r & 3), DIM)];
                if ((w & 0x7F80u) == 0x7F80u) acc.o[i][r] += pt * __uint_as_float((uint32_t)w << 16);
              }
          }
          wave_lds_sync();
        }
      }
    }

    // join the four waves: both halves of a column's sum, then the columns
    acc.l += __shfl_xor(acc.l, 32, 64);
    if (poison) acc.l = __builtin_nanf("");
    if (half == 0) {
      s_ml[wave][col][0] = acc.m;
      s_ml[wave][col][1] = acc.l;
    }
    __syncthreads();
    float m = kFloor, l = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) m = fmaxf(m, s_ml[w][col][0]);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) l += s_ml[w][col][1] * __builtin_amdgcn_exp2f(s_ml[w][col][0] - m);
    const float f = __builtin_amdgcn_exp2f(acc.m - m);
#pragma unroll
    for (int i = 0; i < NB; ++i) acc.o[i] *= f;
    // dims in the order (block, register, half): a lane's place is conflict-free
    auto place = [&](int i, int r) { return ((i * 16 + r) * 2 + half) * 32 + col; };
    if (wave >= 2) {
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) s_o[wave - 2][place(i, r)] = acc.o[i][r];
    }
    __syncthreads();
    if (wave < 2) {
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc.o[i][r] += s_o[wave][place(i, r)];
    }
    __syncthreads();
    if (wave == 1) {
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) s_o[0][place(i, r)] = acc.o[i][r];
    }
    __syncthreads();
    if (wave == 0) {
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) s_o[0][place(i, r)] += acc.o[i][r];
    }
    __syncthreads();

    // the item's rows from s_o[0] (sum m, l in every lane): thread = (row, dims)
    const int nrow = min(kTile, q_rows - first_row);
    const bool split = u0 > 0 || u1 < units;
    auto sum_at = [&](int row, int d) {  // dim d of row `row` in s_o[0]
      const int i = d >> 5, e = d & 31;
      const int r = (e >> 3) * 4 + (e & 3), h = (e >> 2) & 1;
      return s_o[0][((i * 16 + r) * 2 + h) * 32 + row];
    };
    auto out_at = [&](int row) {
      const int q = first_row + row;
      return ((size_t)(v.row0 + q / group) * a.q_heads + kvh * group + q % group) * DIM;
    };
    if (!split) {
      if (wave == 0 && half == 0) s_ml[0][col][1] = l;
      __syncthreads();
      for (int e = tid; e < nrow * (DIM / 2); e += kThreads) {
        const int row = e / (DIM / 2), d = e % (DIM / 2) * 2;
        const float inv = 1.0f / s_ml[0][row][1];
        *reinterpret_cast<uint32_t*>(a.out + out_at(row) + d) = pack_bf16(sum_at(row, d) * inv, sum_at(row, d + 1) * inv);
      }
    } else {
      // hand-off without a device-scope fence (which writes back the whole
      // L2): partials are stored through to the coherent level, every thread
      // waits for its own stores, then one thread counts the arrival
      const int slot = 2 * wg + (at != begin);
      const rsrc_t rp = make_rsrc(a.part + (size_t)slot * (kTile * DIM), kTile * DIM * 4);
      for (int e = tid; e < nrow * (DIM / 4); e += kThreads) {
        const int row = e / (DIM / 4), d = e % (DIM / 4) * 4;
        const u32x4 x = {__float_as_uint(sum_at(row, d)), __float_as_uint(sum_at(row, d + 1)),
                         __float_as_uint(sum_at(row, d + 2)), __float_as_uint(sum_at(row, d + 3))};
        __builtin_amdgcn_raw_buffer_store_b128(x, rp, (row * DIM + d) * 4, 0, kDeviceScope);
      }
      const rsrc_t rm = make_rsrc(a.part_ml, (uint32_t)(2 * a.G) * kTile * 8);
      if (wave == 0 && half == 0) {
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(m), rm, (slot * kTile + col) * 8, 0, kDeviceScope);
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(l), rm, (slot * kTile + col) * 8 + 4, 0, kDeviceScope);
      }
      __atomic_signal_fence(__ATOMIC_SEQ_CST);
      __builtin_amdgcn_s_waitcnt(0);
      __atomic_signal_fence(__ATOMIC_SEQ_CST);
      __syncthreads();
      const int wf = owner_of(item0, total, wgs), wl = owner_of(item0 + units - 1, total, wgs);
      // one counter for each split item: its first unit's workgroup can begin
      // at most one such item before its own end
      if (tid == 0) s_last = atomicAdd(&a.cnt[wf], 1u) == (uint32_t)(wl - wf) ? 1 : 0;
      __syncthreads();
      if (s_last) {
        if (tid == 0) a.cnt[wf] = 0;
        auto slot_of = [&](int w) { return 2 * w + (total * w / wgs < item0 ? 1 : 0); };
        for (int e = tid; e < nrow * (DIM / 4); e += kThreads) {
          const int row = e / (DIM / 4), d = e % (DIM / 4) * 4;
          float M = kFloor;
          for (int w = wf; w <= wl; ++w)
            M = fmaxf(M, __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rm, (slot_of(w) * kTile + row) * 8, 0, kDeviceScope)));
          float L = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
          for (int w = wf; w <= wl; ++w) {
            const int sl = slot_of(w);
            const float mw = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rm, (sl * kTile + row) * 8, 0, kDeviceScope));
            const float lw = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rm, (sl * kTile + row) * 8 + 4, 0, kDeviceScope));
            const rsrc_t rw = make_rsrc(a.part + (size_t)sl * (kTile * DIM), kTile * DIM * 4);
            const u32x4 x = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, (row * DIM + d) * 4, 0, kDeviceScope));
            const float g = __builtin_amdgcn_exp2f(mw - M);
            L += lw * g;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] += __uint_as_float(x[i]) * g;
          }
          const float inv = 1.0f / L;
          *reinterpret_cast<uint2*>(a.out + out_at(row) + d) =
              make_uint2(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv));
        }
      }
    }
    __syncthreads();
    at += u1 - u0;
  }
}

template <int DIM>
hipError_t launch_dim(const AttentionArgs& a, hipStream_t s) {
  if (a.c.kind == 0)
    hipLaunchKernelGGL((kv_attention_kernel<DIM, 0>), dim3(a.G), dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((kv_attention_kernel<DIM, 1>), dim3(a.G), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace

AttentionPlan plan_kv_attention(const KvArgs& c, int num_seq, int total, int q_heads, int num_cu) {
  (void)num_seq; (void)total; (void)q_heads;
  AttentionPlan p{};
  p.G = num_cu * 2;
  p.max_items = p.G;
  p.off_part = ((size_t)p.G * 4 + 255) & ~size_t(255);
  p.off_ml = p.off_part + (size_t)2 * p.G * kTile * c.dim * 4;
  p.ws_bytes = p.off_ml + (size_t)2 * p.G * kTile * 8;
  return p;
}

hipError_t launch_kv_attention(const AttentionArgs& a, hipStream_t s) {
  switch (a.c.dim) {
    case 64: return launch_dim<64>(a, s);
    case 128: return launch_dim<128>(a, s);
    default: return launch_dim<256>(a, s);
  }
}

}  // namespace w12
