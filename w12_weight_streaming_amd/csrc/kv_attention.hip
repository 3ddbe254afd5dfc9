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
// Work split: a sequence's query rows (row x head of the group) are cut into
// tiles of 32, a block is the tiles of WR = 1, 2 or 4 waves, and the
// workgroup's eight waves walk 8 / WR groups of 32 tokens at a time (a step). An
// item is (sequence, kv head, block), its steps run over the pages, then the
// recent rows. The steps of all items in order are cut into equal runs, one for
// each workgroup, so ragged batches balance. Items that several workgroups share
// leave partial sums, which a second launch joins in workgroup order: results
// are bitwise reproducible.
//
// What bounds it, as measured:
// - 32 sequences of one row, 16384 tokens, 8 x 6 heads of 128: 95 us for 526 MB,
//   5.5 TB/s of HBM reads (a large copy moves 4.8);
// - 24 trees of 8 rows, 8191 tokens, int8: 67 us for 232 MB, 3.5 TB/s: items of
//   1.3 runs each, whose beginnings and ends (queries, recent rows, the waves'
//   join, partial sums) take some 20 us in which few pages are under way;
// - a 32-row tree, 32000 tokens, 4 x 6 heads of 256: 55 us for 66 MB and 25
//   GFLOP, of which the join takes 10. The wave of each of its six tiles loads and
//   converts every page for itself: vector instructions take 41% of a SIMD's time,
//   matrix instructions 29%, and waves wait for loads 36% of theirs (registers hold
//   the next step's pages only);
// - 512 prompt rows, 16 x 6 heads of 64: 94 us for 54.8 GFLOP, 584 TFLOP/s:
//   exponentials, conversions and packing (a product of 64 dims is short against
//   the 16 probabilities a lane makes for it). Vector instructions take 65% of a
//   SIMD's time, matrix instructions 27%, hardly ever at once;
// - one row over 700 tokens: 14 us and 4 for the join, 1.6 MB: chains of dependent
//   loads (offsets, slot, length, page table, scales, keys), barriers, two launches.
#include <limits.h>

#include "kv_internal.h"
#include "w12_device.h"

namespace w12 {
namespace {

constexpr int kThreads = 512, kWaves = 8;  // one workgroup a CU, two waves a SIMD
constexpr int kTile = 32;        // query rows of a tile
constexpr int kPartFloats = 16384;  // floats of one partial sum: a block's rows x dims, at most
// steps that an item's beginning and end are worth (queries, the first pages'
// chain of loads, recent rows, the join of the waves): they count as its last
// steps, in which nothing is done (3, 6 and 10 of them: batch decode 100, 95 and
// 97 us; 24 trees of 8 rows 74, 71 and 71)
constexpr int kItemSteps = 6;
constexpr float kLog2e = 1.44269504088896340736f;
// a new maximum is taken when a score passes the running one by this much
// (in powers of two): until then probabilities may reach 2^8, which neither
// fp32 sums nor bf16 operands lose anything by, and the rescaling is skipped
// (512 prompt rows: 96 us, 101 with a new maximum for every higher score)
constexpr float kSlack = 8.0f;
constexpr float kFloor = -3.402823466e38f;  // running maximum before the first score

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {  // one v_cvt_pk_bf16_f32
  bf16x2 v;
  v[0] = (__bf16)a;
  v[1] = (__bf16)b;
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ bf16x8 as_operand(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(bf16x8, u32x4{a, b, c, d});
}

// Four 8-bit codes as bf16 pairs, exactly.
template <int KIND>
__device__ __forceinline__ void codes4(uint32_t x, uint32_t& lo, uint32_t& hi) {
  // opaque: else the compiler carries loaded codes from one step to the next
  // byte by byte, in a register each
  asm("" : "+v"(x));
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

// All ones where bit b of x is set (masks as values: as conditions they would
// take a pair of scalar registers each).
__device__ __forceinline__ uint32_t bit_mask(uint32_t x, int b) { return (uint32_t)((int32_t)(x << (31 - b)) >> 31); }

// The larger of a lane's value and that of its other half.
__device__ __forceinline__ float exchange_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// U groups of 32 scores per row, x = sc * c in powers of two (only where
// `see` has the token's bit, if MASK; a group that `valid` leaves out counts
// for nothing). The probabilities come out times the value scale 2^lv, as the
// product's operands; their sum without it (times rv = 2^-lv) joins l. The sum
// is taken over the operands as rounded, two at a time.
// The operands are one bf16 each, off by up to 2^-8 of a probability: values
// and codes are then multiplied at the full rate. As two bf16 each (a probability
// and what its rounding left, a second product) outputs are the 64-bit ones
// rounded, at 17.9 us for 17.1 (one row), 96.5 for 94.9 (batch decode), 60.9 for
// 55.5 (the tree), 80.2 for 71.3 (24 trees), 127.6 for 97.6 (prompt). With one, the
// outputs' error (2-norms over the result's) is 1.04 to 1.35 times what rounding the
// output alone makes, 0.9e-3 to 1.7e-3.
template <int NB, int U, bool MASK>
__device__ __forceinline__ void softmax_step(f32x16 (&o)[NB], float& m, float& l, f32x16 (&sc)[U], const float (&c)[U],
                                             const float (&lv)[U], const float (&rv)[U], const bool (&valid)[U],
                                             uint32_t see, int half, bf16x8 (&pb)[U][2]) {
  float mx = kFloor;
  const uint32_t mine = see >> (half * 4);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float x = kFloor;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      if (MASK) {
        const uint32_t keep = bit_mask(mine, (r >> 2) * 8 + (r & 3));
        sc[u][r] = __uint_as_float((__float_as_uint(sc[u][r]) & keep) | (0xFF800000u & ~keep));
      }
      x = fmaxf(x, sc[u][r]);
    }
    if (valid[u]) mx = fmaxf(mx, x * c[u]);
  }
  mx = exchange_max(mx);
  if (__any(mx > m + kSlack)) {
    const float nm = fmaxf(m, mx);
    const float al = __builtin_amdgcn_exp2f(m - nm);
    m = nm;
    l *= al;
#pragma unroll
    for (int i = 0; i < NB; ++i) o[i] *= al;
  }
  constexpr uint32_t kOnes = 0x3F803F80u;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const float base = lv[u] - m;
    uint32_t w[8];
    float sum = 0.f;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      w[r] = pack_bf16(__builtin_amdgcn_exp2f(__builtin_fmaf(sc[u][2 * r], c[u], base)),
                       __builtin_amdgcn_exp2f(__builtin_fmaf(sc[u][2 * r + 1], c[u], base)));
      sum = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w[r]), __builtin_bit_cast(bf16x2, kOnes), sum, false);
    }
    l = __builtin_fmaf(sum, rv[u], l);
    pb[u][0] = as_operand(w[0], w[1], w[2], w[3]);
    pb[u][1] = as_operand(w[4], w[5], w[6], w[7]);
  }
}

// Most tiles of a block. More of them read a page for more rows but split the
// tokens among fewer waves; at one workgroup a CU the pages come from the caches
// the second time, so few tiles win (512 prompt rows, 64-dim heads: 97 us with up
// to 2 or 8 tiles, 94 with 4; 128 dims: 84, 86 with 4).
template <int DIM>
constexpr int kBlockTiles = DIM == 64 ? 4 : 2;

// Waves along the rows for n tiles: `most`, unless that leaves over a seventh of
// them idle (6 tiles of 128 dims over 8192 tokens: 39 us as 4 + 2, 30 by twos).
__device__ __forceinline__ int waves_along_rows(int n, int most) {
  int wr = most;
  while (wr > 1 && (n <= wr / 2 || ((n + wr - 1) / wr * wr - n) * 7 > n)) wr >>= 1;
  return wr;
}

// What the join needs to know of the item that a workgroup begins and others
// go on with.
struct SplitItem {
  int last;             // its last workgroup, -1: none
  int rows;             // query rows
  int row0, first_row;  // first row of the sequence; first query row of the item
  int kvh, first_slot;  // partial slot of the first workgroup: 0 or 1
};

// A sequence as the scan found it.
struct SeqInfo {
  int len;     // -1: refused
  int slot;
  short row0, rows;
};

template <int DIM>
struct Shared {
  static constexpr int kRows = kBlockTiles<DIM> * kTile;
  union {
    uint4 q[kBlockTiles<DIM>][DIM / 32][2][64];  // query tiles as B operands
    float4 x[kWaves][512];                       // sums that waves hand to each other
  };
  uint32_t anc[kRows][kStepRows / 32];
  int64_t first[kStepRows + 1];  // steps before each sequence
  SeqInfo seq[kStepRows];
  int parent[kStepRows];
  float ml[kWaves][kTile][2];
  int64_t scan[kWaves];
  int bad, strange;
};

template <int DIM, int KIND, bool STREAM>
__global__ __launch_bounds__(kThreads, 2) void kv_attention_kernel(AttentionArgs a) {
  constexpr int NB = DIM / 32;
  constexpr int U = DIM == 256 ? 1 : 2;       // groups of 32 tokens a wave takes at a time
  constexpr bool kQueryRegs = DIM <= 128;     // its query operands stay in registers
  __shared__ Shared<DIM> sh;
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int group = a.q_heads / a.c.kv_heads, per_page = a.c.page / kGroup;
  SplitItem* split_item = static_cast<SplitItem*>(a.items) + blockIdx.x;

  // steps of every sequence, then their running sum
  struct Shape {
    int wr, blocks, page_units, steps;
  };
  auto shape_of = [&](const SeqInfo& v) __attribute__((always_inline)) {
    Shape h;
    const int tiles = (v.rows * group + kTile - 1) / kTile;
    h.wr = waves_along_rows(tiles, a.most_tiles);
    h.blocks = (tiles + h.wr - 1) / h.wr;
    const int full = v.len / a.c.page, tail = v.len - full * a.c.page;
    h.page_units = v.len < 0 ? 0 : full * per_page;
    const int units = v.len < 0 ? 1 : h.page_units + (tail + v.rows + kGroup - 1) / kGroup;
    const int wt = kWaves / h.wr;
    h.steps = (units + wt - 1) / wt + kItemSteps;
    return h;
  };
  {
    static_assert(kThreads == kStepRows);
    int64_t mine = 0;
    SeqView v{};
    int back = 0;
    if (tid < a.st.num_seq) {
      v = seq_view(a.c, a.st, tid);
      back = a.st.row_off[tid] > a.st.row_off[tid + 1];
    }
    if (__syncthreads_or(back))  // only then can two sequences share rows
      for (int j = 0; j < tid && tid < a.st.num_seq; ++j)
        if (rows_meet(a.st.row_off, a.st.total, j, v.row0, v.rows)) v.rows = 0;
    if (tid < a.st.num_seq) {
      SeqInfo n;
      n.len = v.ok ? v.len : -1;
      n.slot = v.slot;
      n.row0 = (short)v.row0;
      n.rows = (short)v.rows;
      sh.seq[tid] = n;
      const Shape h = shape_of(n);
      mine = (int64_t)h.blocks * a.c.kv_heads * h.steps;
    }
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint32_t lo = __shfl_up((uint32_t)upto, o, 64), hi = __shfl_up((uint32_t)((uint64_t)upto >> 32), o, 64);
      if (lane >= o) upto += (int64_t)(((uint64_t)hi << 32) | lo);
    }
    if (lane == 63) sh.scan[wave] = upto;
    __syncthreads();
    for (int w = 0; w < wave; ++w) upto += sh.scan[w];
    sh.first[tid] = upto - mine;
    if (tid == kThreads - 1) sh.first[kStepRows] = upto;
  }
  if (tid == 0) split_item->last = -1;
  __syncthreads();
  const int64_t total = sh.first[kStepRows];
  const int wgs = (int)min((int64_t)a.G, total);
  const int wg = blockIdx.x;
  if (wg >= wgs) return;
  const int64_t begin = total * wg / wgs, end = total * (wg + 1) / wgs;

  int seq;  // the first sequence whose steps reach past `begin`
  {
    int lo = 0, hi = a.st.num_seq - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (sh.first[mid + 1] > begin) hi = mid; else lo = mid + 1;
    }
    seq = lo;
  }

  // the thread's index, opaque: each phase of an item derives its places anew,
  // so that none is computed ahead and kept in a register (or spilled) through
  // the others
  auto own_index = [thread = tid]() __attribute__((always_inline)) {
    int t = thread;
    asm volatile("" : "+v"(t));
    return t;
  };
  for (int64_t at = begin; at < end;) {
    const int tid = own_index(), lane = tid & 63, col = lane & 31, half = lane >> 5;
    while (sh.first[seq + 1] <= at) ++seq;
    const SeqInfo v = sh.seq[seq];
    const Shape h = shape_of(v);
    const bool ok = v.len >= 0;
    const int tail = ok ? v.len - h.page_units * kGroup : 0;
    const int item = (int)((at - sh.first[seq]) / h.steps);
    const int64_t item0 = sh.first[seq] + (int64_t)item * h.steps;  // the item's first step
    const int st0 = (int)(at - item0), st1 = (int)min((int64_t)h.steps, end - item0);
    const int second = at != begin;  // the run's second partial sum
    at += st1 - st0;
    if (st0 >= h.steps - kItemSteps) continue;
    const int kvh = item / h.blocks, block = item % h.blocks;
    const int wt = kWaves / h.wr, wr = wave & (h.wr - 1), ph = wave / h.wr;  // the wave's tiles, its share of the tokens
    const int block_row = block * h.wr * kTile, q_rows = v.rows * group;
    const int block_rows = min(h.wr * kTile, q_rows - block_row);
    const int wave_row = block_row + wr * kTile;  // the wave's first query row
    const bool idle = wave_row >= q_rows || !ok;
    const int b_lo = block_row / group, b_hi = min((int)v.rows, (block_row + block_rows - 1) / group + 1);
    const int my = wave_row + col;  // the lane's query row: row my / group, head my % group
    const bool on = my < q_rows && ok;

    // the tile's query rows as B operands: dims 32 i + 16 half + 0..15 of a lane's row
    bf16x8 qr[kQueryRegs ? NB : 1][2];
    __syncthreads();  // the last item's joins are done with the shared arrays
    if (kQueryRegs || ph == 0) {
      const int r = on ? my / group : 0, hd = kvh * group + (on ? my % group : 0);
      const u32x4* p = reinterpret_cast<const u32x4*>(a.q + ((size_t)(v.row0 + r) * a.q_heads + hd) * DIM + half * 16);
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          u32x4 x = {0, 0, 0, 0};
          if (on) x = p[i * 4 + e];
          if constexpr (kQueryRegs)
            qr[i][e] = __builtin_bit_cast(bf16x8, x);
          else
            sh.q[wr][i][e][lane] = __builtin_bit_cast(uint4, x);
        }
    }
    // pages: units st * wt + ph, ids and scales of 64 at a time
    const int pst1 = idle ? st0 : min(st1, (h.page_units - ph + wt - 1) / wt);
    const int np = max(0, pst1 - st0);
    const uint8_t* page0 = a.c.pages + page_at(a.c, a.layer, 0, kvh, 0);
    const size_t page_bytes = (size_t)a.c.kv_heads * 2 * a.c.page * DIM;
    const int to_v = a.c.page * DIM;
    const float c2 = a.scale * kLog2e;
    int id, off, cnt;
    float ks, lv, rv;
    // ids of up to 64 units, a lane each, and (as loaded) their scales
    auto fetch = [&](int kb, int lane) __attribute__((always_inline)) {
      cnt = min(64, np - kb);
      id = off = 0;
      if (lane < cnt) {
        const int u = (st0 + kb + lane) * wt + ph, j = u / per_page;
        id = a.c.table[(size_t)v.slot * a.c.max_pages + j];
        off = (u - j * per_page) * (kGroup * DIM);
      }
      const bool good = id >= 0 && id < a.c.num_pages;
      if (!good) id = 0;
      const float2 sc = *reinterpret_cast<const float2*>(a.c.scales + scale_at(a.c, a.layer, id, kvh, 0));
      ks = sc.x;
      rv = sc.y;
      off = good ? off : off | INT_MIN;
    };
    // the scales' factors; lanes past the last unit: a weight of zero (2^-inf)
    auto factors = [&](int lane) __attribute__((always_inline)) {
      const bool live = lane < cnt;
      ks = live ? ks * c2 : 0.f;
      if (off < 0) ks = __builtin_nanf("");
      lv = live ? __builtin_amdgcn_logf(rv) : -__builtin_huge_valf();
      rv = live ? __builtin_amdgcn_rcpf(rv) : 0.f;
    };
    // past the last unit the loads repeat it: they stay unconditional, so
    // that every wait is for the oldest ones in flight alone
    auto at_page = [&](int k) __attribute__((always_inline)) {
      k = min(k, cnt - 1);
      const uint32_t pid = __builtin_amdgcn_readlane(id, k), o = __builtin_amdgcn_readlane(off, k) & INT_MAX;
      return page0 + (size_t)pid * page_bytes + o;
    };
    auto load_page = [&](const uint8_t* p, int to, u32x4 (&x)[NB]) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const u32x4* q = reinterpret_cast<const u32x4*>(p + i * 1024 + to);
        x[i] = STREAM ? __builtin_nontemporal_load(q) : *q;
      }
    };
    u32x4 kr[U][NB], vr[U][NB];
    // the first keys are on their way before anything else of the item,
    // where the registers hold them next to the recent rows' operands
    auto load_keys = [&](int to) __attribute__((always_inline)) {
#pragma unroll
      for (int u = 0; u < U; ++u) load_page(at_page(u), to, kr[u]);
    };
    auto load_values = [&](int to) __attribute__((always_inline)) {
#pragma unroll
      for (int u = 0; u < U; ++u) load_page(at_page(u) + to_v, to, vr[u]);
    };
    if (np > 0) {
      fetch(0, lane);
      if constexpr (DIM <= 128) load_keys(lane * 16);
    }

    // ancestors of the block's rows, a set of bits for each
    if (tid == 0) sh.bad = sh.strange = 0;
    __syncthreads();
    if (ok && st1 * wt > h.page_units) {
      if (a.st.parent) {
        int bad = 0;
        for (int i = tid; i < v.rows; i += kThreads) {
          const int p = a.st.parent[v.row0 + i];
          sh.parent[i] = p;
          if (i == 0 ? p != -1 : (p < 0 || p >= i)) bad = 1;
        }
        for (int i = tid; i < (b_hi - b_lo) * (kStepRows / 32); i += kThreads) (&sh.anc[0][0])[i] = 0;
        if (bad) sh.bad = 1;
        __syncthreads();
        if (!sh.bad)
          for (int r = b_lo + tid; r < b_hi; r += kThreads)
            for (int i = r; i >= 0; i = sh.parent[i]) sh.anc[r - b_lo][i >> 5] |= 1u << (i & 31);
      } else {
        for (int i = tid; i < (b_hi - b_lo) * (kStepRows / 32); i += kThreads) {
          const int r = b_lo + i / (kStepRows / 32) - (i % (kStepRows / 32)) * 32;  // highest visible bit
          (&sh.anc[0][0])[i] = r < 0 ? 0u : r >= 31 ? ~0u : (2u << r) - 1u;
        }
      }
    }
    __syncthreads();
    const bool poison = !ok || sh.bad;

    f32x16 acc[NB];
    float m = kFloor, l = 0.f;
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][r] = 0.f;
    // recent rows: the committed tail, then the step's rows; the wave's tiles
    // see nothing behind their own last row
    if (!poison && !idle) {
      const int lane = own_index() & 63, col = lane & 31, half = lane >> 5, my = wave_row + col;
      const bool on = my < q_rows;
      const uint4* qs = &sh.q[wr][0][0][lane];
      auto query = [&](int i, int e) __attribute__((always_inline)) {
        if constexpr (kQueryRegs)
          return qr[i][e];
        else
          return __builtin_bit_cast(bf16x8, qs[(i * 2 + e) * 64]);
      };
      const uint16_t* kb = a.c.recent + recent_at(a.c, a.layer, v.slot, kvh, 0) + lane * 16;
      const uint16_t* vb = a.c.recent + recent_at(a.c, a.layer, v.slot, kvh, 1) + lane * 16;
      const int rows = tail + v.rows, seen = tail + min((int)v.rows, (wave_row + kTile - 1) / group + 1);
      const uint32_t* anc = sh.anc[on ? my / group - b_lo : 0];
      constexpr int HB = NB < 4 ? NB : 4;  // blocks of 32 dims loaded at a time
      auto load = [&](const uint16_t* p, u32x4 (&x)[HB][2]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < HB; ++i) {
          x[i][0] = *reinterpret_cast<const u32x4*>(p + i * 1024);
          x[i][1] = *reinterpret_cast<const u32x4*>(p + i * 1024 + 8);
        }
      };
      for (int st = max(st0, (h.page_units - ph + wt - 1) / wt); st < st1; ++st) {
        const int t0 = (st * wt + ph - h.page_units) * kGroup;
        if (t0 >= seen) break;
        const int held = min(32, rows - t0);  // rows of this group that there are
        const uint32_t there = held == 32 ? ~0u : (1u << held) - 1u;
        const uint16_t* kp = kb + (size_t)t0 * DIM;
        const uint16_t* vp = vb + (size_t)t0 * DIM;
        u32x4 x[HB][2];
        f32x16 sc[1];
#pragma unroll
        for (int r = 0; r < 16; ++r) sc[0][r] = 0.f;
        load(kp, x);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i0 = 0; i0 < NB; i0 += HB) {
          if (i0) load(kp + i0 * 1024, x);
#pragma unroll
          for (int i = 0; i < HB; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              sc[0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x[i][e]), query(i0 + i, e), sc[0], 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
        }
        load(vp, x);
        // bit b: the lane's row sees place t0 + b: every tail token, and its ancestors
        uint32_t see = 0;
        if (on) {
          const int shift = t0 - tail;  // the step's row at place t0
          if (shift >= 0) {
            const int k = shift >> 5, b = shift & 31;
            const uint64_t two = (uint64_t)anc[k] | ((uint64_t)(k + 1 < kStepRows / 32 ? anc[k + 1] : 0u) << 32);
            see = (uint32_t)(two >> b);
          } else if (shift > -32) {
            see = (anc[0] << -shift) | ((1u << -shift) - 1u);
          } else {
            see = ~0u;
          }
          see &= there;
        }
        bf16x8 pb[1][2];
        softmax_step<NB, 1, true>(acc, m, l, sc, {c2}, {0.f}, {1.f}, {true}, see, half, pb);
        // values: what a query row does not see, be it an infinity or NaN of
        // another branch or whatever lies behind the rows, must not meet its
        // probability of zero; finite values may
        const uint32_t mine = there >> (half * 4);
        uint32_t odd = 0;
#pragma unroll
        for (int i0 = 0; i0 < NB; i0 += HB) {
          if (i0) load(vp + i0 * 1024, x);
          uint32_t any = 0;  // an exponent of all ones carries into the sign's place
#pragma unroll
          for (int i = 0; i < HB; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) any |= (x[i][e >> 2][e & 3] & 0x7F807F80u) + 0x00800080u;
          if (__any(any & 0x80008000u)) {
#pragma unroll
            for (int i = 0; i < HB; ++i)
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                // slots 2 e, 2 e + 1: tokens 8 (e >> 1) + 4 half + 2 (e & 1) and the next
                const int b = (e >> 1) * 8 + (e & 1) * 2;
                uint32_t w = x[i][e >> 2][e & 3];
                w &= (bit_mask(mine, b) & 0xFFFFu) | (bit_mask(mine, b + 1) & 0xFFFF0000u);
                const uint32_t bad = ((((w & 0x7F807F80u) + 0x00800080u) >> 15) & 0x00010001u) * 0xFFFFu;
                odd |= bad;
                w &= ~bad;
                x[i][e >> 2][e & 3] = w;
              }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < HB; ++i)
              acc[i0 + i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x[i][e]), pb[0][e], acc[i0 + i], 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
        }
        if (odd) sh.strange = 1;
      }
    }

    for (int kb = 0; kb < np;) {
      const int lane = own_index() & 63, half = lane >> 5, to = lane * 16;
      if (kb) fetch(kb, lane);
      if (kb || DIM > 128) load_keys(to);
      load_values(to);
      factors(lane);
      const uint4* qs = &sh.q[wr][0][0][lane];
      auto query = [&](int i, int e) __attribute__((always_inline)) {
        if constexpr (kQueryRegs)
          return qr[i][e];
        else
          return __builtin_bit_cast(bf16x8, qs[(i * 2 + e) * 64]);
      };
      for (int k = 0; k < cnt; k += U) {
        f32x16 sc[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int r = 0; r < 16; ++r) sc[u][r] = 0.f;
        bf16x8 q0 = query(0, 0), q1 = query(0, 1);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          // the next operands' reads are under way while these are used
          const bf16x8 n0 = query(i + 1 < NB ? i + 1 : i, 0), n1 = query(i + 1 < NB ? i + 1 : i, 1);
          bf16x8 x[U], y[U];
#pragma unroll
          for (int u = 0; u < U; ++u) codes16<KIND>(kr[u][i], x[u], y[u]);
          if constexpr (!kQueryRegs) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int u = 0; u < U; ++u) sc[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[u], q0, sc[u], 0, 0, 0);
#pragma unroll
          for (int u = 0; u < U; ++u) sc[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(y[u], q1, sc[u], 0, 0, 0);
          q0 = n0;
          q1 = n1;
          // in order: the next fragments' conversion runs under these
          // products, and no earlier (hoisted, they take every register)
          __builtin_amdgcn_sched_barrier(0);
        }
        const uint8_t* next[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          next[u] = at_page(k + U + u);
          load_page(next[u], to, kr[u]);
        }
        float c[U], e[U], f[U];
        bool valid[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          auto lane_of = [&](float x) __attribute__((always_inline)) {
            return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), k + u));
          };
          c[u] = lane_of(ks);
          e[u] = lane_of(lv);
          f[u] = lane_of(rv);
          valid[u] = k + u < cnt;
        }
        bf16x8 pb[U][2];
        softmax_step<NB, U, false>(acc, m, l, sc, c, e, f, valid, 0u, half, pb);
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
          for (int i = 0; i < NB; i += 2) {
            bf16x8 x[2], y[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) codes16<KIND>(vr[u][i + j], x[j], y[j]);
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[i + j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[j], pb[u][0], acc[i + j], 0, 0, 0);
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[i + j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(y[j], pb[u][1], acc[i + j], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) load_page(next[u] + to_v, to, vr[u]);
      }
      kb += 64;
    }

    // join the waves that share a tile: both halves of a column's sum, then
    // the waves' shares of the tokens
    {
    const int tid = own_index(), lane = tid & 63, col = lane & 31, half = lane >> 5, my = wave_row + col;
    l += __shfl_xor(l, 32, 64);
    if (poison) l = __builtin_nanf("");
    if (half == 0) {
      sh.ml[wave][col][0] = m;
      sh.ml[wave][col][1] = l;
    }
    __syncthreads();
    constexpr int kR = 16 * NB;
    float r[kR];  // the lane's sums, now one by one (a change of one in a vector of 16 may copy it)
    {
      const float own = m;
      for (int w = wr; w < kWaves; w += h.wr) m = fmaxf(m, sh.ml[w][col][0]);
      l = 0.f;
      for (int w = wr; w < kWaves; w += h.wr) l += sh.ml[w][col][1] * __builtin_amdgcn_exp2f(sh.ml[w][col][0] - m);
      const float scale = __builtin_amdgcn_exp2f(own - m);
#pragma unroll
      for (int f = 0; f < kR; ++f) r[f] = acc[f >> 4][f & 15] * scale;
    }
    // Of a tile's kR = 16 NB sums a lane, each of its wt waves ends with
    // kR / wt: in every round two waves swap halves of what they hold, each
    // adding the half that it keeps. Sum F is dim 2 F + 4 half (F % 4 == 0).
    int mine0 = 0;  // the wave's first sum
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      constexpr int kMost = 32;  // sums of a lane in the exchange buffer
      const int n = kR >> (j + 1), part_n = n < kMost ? n : kMost, stride = kWaves >> (j + 1);  // partner: ph ^ stride
      if (stride < h.wr) break;
      const bool upper = tid & (stride * 64);  // keeps the upper half
      if (wave & stride) mine0 += n;
#pragma unroll
      for (int f0 = 0; f0 < n; f0 += part_n) {
#pragma unroll
        for (int f = f0; f < f0 + part_n; ++f) {  // selects, not a branch: that would hold every sum twice
          const float x = r[f], y = r[f + n];
          r[f] = upper ? y : x;
          r[f + n] = upper ? x : y;
        }
        __builtin_amdgcn_sched_barrier(0);
        float4* give = sh.x[wave] + lane;
        const float4* take = sh.x[wave ^ stride] + lane;
#pragma unroll
        for (int f = 0; f < part_n; f += 4)
          give[f * 16] = make_float4(r[n + f0 + f], r[n + f0 + f + 1], r[n + f0 + f + 2], r[n + f0 + f + 3]);
        __syncthreads();
#pragma unroll
        for (int f = 0; f < part_n; f += 4) {
          const float4 t = take[f * 16];
          r[f0 + f] += t.x;
          r[f0 + f + 1] += t.y;
          r[f0 + f + 2] += t.z;
          r[f0 + f + 3] += t.w;
        }
        __syncthreads();
      }
    }
    // out, or to the partial sums
    const bool split = st0 > 0 || st1 < h.steps - kItemSteps;
    float* part = a.part + (size_t)(2 * wg + second) * kPartFloats;
    float2* part_ml = reinterpret_cast<float2*>(a.part_ml) + (size_t)(2 * wg + second) * (kPartFloats / DIM);
    if (my < q_rows) {
      const int row = my - block_row, n = kR / wt;
      if (!split) {
        const float inv = 1.0f / l;
        uint16_t* o = a.out + ((size_t)(v.row0 + my / group) * a.q_heads + kvh * group + my % group) * DIM + 2 * mine0 + half * 4;
#pragma unroll
        for (int f = 0; f < kR; f += 4)
          if (f < n)
            *reinterpret_cast<uint2*>(o + 2 * f) =
                make_uint2(pack_bf16(r[f] * inv, r[f + 1] * inv), pack_bf16(r[f + 2] * inv, r[f + 3] * inv));
      } else {
        float* o = part + row * DIM + 2 * mine0 + half * 4;
#pragma unroll
        for (int f = 0; f < kR; f += 4)
          if (f < n) *reinterpret_cast<float4*>(o + 2 * f) = make_float4(r[f], r[f + 1], r[f + 2], r[f + 3]);
        if (half == 0 && ph == 0) part_ml[row] = make_float2(m, l);
      }
    }
    // infinities and NaN among the run's recent values, by themselves, for the
    // rows that see them: no finite sum brings the output back from them
    if (sh.strange) {
      __syncthreads();
      const uint16_t* vb = a.c.recent + recent_at(a.c, a.layer, v.slot, kvh, 1);
      const int t0 = max(0, (st0 * wt - h.page_units) * kGroup);
      const int t1 = min(tail + v.rows, (st1 * wt - h.page_units) * kGroup);
      for (int e = tid; e < block_rows * DIM; e += kThreads) {
        const int q = block_row + e / DIM, d = e % DIM, r = q / group;
        float sum = 0.f;
        for (int t = t0; t < t1; ++t) {
          const int j = t - tail;
          const uint16_t w = vb[value_at(t, d, DIM)];
          if ((w & 0x7F80u) == 0x7F80u && (j < 0 || ((sh.anc[r - b_lo][j >> 5] >> (j & 31)) & 1)))
            sum += __uint_as_float((uint32_t)w << 16);
        }
        if (sum == 0.f) continue;
        if (split) {
          part[e] += sum;
        } else {
          uint16_t* o = a.out + ((size_t)(v.row0 + r) * a.q_heads + kvh * group + q % group) * DIM + d;
          *o = f32_to_bf16_rne(__uint_as_float((uint32_t)*o << 16) + sum);
        }
      }
    }
    if (split && st0 == 0 && tid == 0) {  // at most one item per workgroup begins here and ends elsewhere
      SplitItem t;
      t.last = (int)(((item0 + h.steps - kItemSteps) * wgs - 1) / total);
      t.rows = block_rows;
      t.row0 = v.row0;
      t.first_row = block_row;
      t.kvh = kvh;
      t.first_slot = second;
      *split_item = t;
    }
    }
  }
}

// Joins the partial sums of the items that several workgroups share: with
// the largest running maximum M, out = sum_w 2^(m_w - M) o_w / sum_w 2^(m_w - M) l_w.
// One workgroup per split item and piece of its rows. The weights 2^(m_w - M)
// of its rows come first, a thread each; then a thread owns 4 dims of a row,
// its loads from the contributors independent of each other. Bound by latency:
// 4 to 10 us, of which an empty launch is 3. Tried: 8 pieces a row set (the tree of
// 256 dims +6 us), contributors shared among 2 or 4 times the threads (+4, +13).
constexpr int kJoinThreads = 256, kJoinPieces = 16;

template <int DIM>
__global__ __launch_bounds__(kJoinThreads) void kv_attention_join_kernel(AttentionArgs a) {
  constexpr int kPer = DIM / 4;               // threads of a row
  constexpr int kRows = kJoinThreads / kPer;  // rows a workgroup handles at a time
  constexpr int kFew = 64;                    // contributors whose weights are kept at a time
  __shared__ float s_w[kRows][kFew], s_m[kRows][kPer], s_l[kRows][kPer];
  const SplitItem t = static_cast<const SplitItem*>(a.items)[blockIdx.x];
  if (t.last < 0) return;
  const int group = a.q_heads / a.c.kv_heads, wf = blockIdx.x, n = t.last - wf + 1;
  const int r = threadIdx.x / kPer, d4 = threadIdx.x % kPer;
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml);
  for (int row0 = blockIdx.y * kRows; row0 < t.rows; row0 += kJoinPieces * kRows) {
    const int row = min(row0 + r, t.rows - 1);
    // contributor w's partial sum: the first may be its workgroup's second, later ones begin with the item
    auto slot = [&](int w) __attribute__((always_inline)) { return 2 * (wf + w) + (w ? 0 : t.first_slot); };
    auto ml_at = [&](int w) __attribute__((always_inline)) { return ml[(size_t)slot(w) * (kPartFloats / DIM) + row]; };
    float M = kFloor;
    for (int w = d4; w < n; w += kPer) M = fmaxf(M, ml_at(w).x);
    s_m[r][d4] = M;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) M = fmaxf(M, s_m[r][i]);
    float L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w0 = 0; w0 < n; w0 += kFew) {
      const int cnt = min(kFew, n - w0);
      __syncthreads();
      for (int w = d4; w < cnt; w += kPer) {
        const float2 x = ml_at(w0 + w);
        const float g = __builtin_amdgcn_exp2f(x.x - M);
        s_w[r][w] = g;
        L += x.y * g;
      }
      __syncthreads();
#pragma unroll 8
      for (int w = 0; w < cnt; ++w) {
        const float4 z = *reinterpret_cast<const float4*>(a.part + (size_t)slot(w0 + w) * kPartFloats + row * DIM + d4 * 4);
        const float g = s_w[r][w];
        o.x = __builtin_fmaf(z.x, g, o.x);
        o.y = __builtin_fmaf(z.y, g, o.y);
        o.z = __builtin_fmaf(z.z, g, o.z);
        o.w = __builtin_fmaf(z.w, g, o.w);
      }
    }
    s_l[r][d4] = L;
    __syncthreads();
    L = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) L += s_l[r][i];
    if (row0 + r < t.rows) {
      const float inv = 1.0f / L;
      const int q = t.first_row + row;
      *reinterpret_cast<uint2*>(a.out + ((size_t)(t.row0 + q / group) * a.q_heads + t.kvh * group + q % group) * DIM + d4 * 4) =
          make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
    }
  }
}

template <int DIM, bool STREAM>
hipError_t launch_dim(const AttentionArgs& a, hipStream_t s) {
  if (a.c.kind == 0)
    hipLaunchKernelGGL((kv_attention_kernel<DIM, 0, STREAM>), dim3(a.G), dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((kv_attention_kernel<DIM, 1, STREAM>), dim3(a.G), dim3(kThreads), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((kv_attention_join_kernel<DIM>), dim3(a.G, kJoinPieces), dim3(kJoinThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace

AttentionPlan plan_kv_attention(const KvArgs& c, int num_cu) {
  AttentionPlan p{};
  p.G = num_cu;
  p.off_part = ((size_t)p.G * sizeof(SplitItem) + 255) & ~size_t(255);
  p.off_ml = p.off_part + (size_t)2 * p.G * kPartFloats * 4;
  p.ws_bytes = p.off_ml + (size_t)2 * p.G * (kPartFloats / c.dim) * 8;
  return p;
}

hipError_t launch_kv_attention(const AttentionArgs& in, hipStream_t s) {
  AttentionArgs a = in;
  const int64_t rows = (int64_t)a.st.total * (a.q_heads / a.c.kv_heads);
  // Items that four or more workgroups share are cut into single tiles: their
  // pages' second readings are cache hits, and a partial sum is half as large (a
  // 32-node tree over 32000 tokens, 6 tiles of 256 dims: 59 -> 53 us; of 128
  // dims over 8192 tokens: 30 -> 25). Where items fill the card, single tiles cost
  // re-reading (8 trees of 4 tiles over 16000 tokens: 56 -> 77).
  const bool few = (rows + kTile - 1) / kTile * a.c.kv_heads * 4 <= a.G;
  a.most_tiles = few ? 1 : a.c.dim == 64 ? 4 : 2;
  // Sequences whose rows make one block read every page once: past the caches
  // (batch decode 105 -> 95 us, 24 trees of 2 tiles 70 -> 65), unless more than two
  // waves share the loads, or two that hold 256 dims and so drift apart (49 -> 55).
  const bool stream = rows <= (int64_t)a.st.num_seq * kTile * (few || a.c.dim == 256 ? 1 : 2);
  switch (a.c.dim) {
    case 64: return stream ? launch_dim<64, true>(a, s) : launch_dim<64, false>(a, s);
    case 128: return stream ? launch_dim<128, true>(a, s) : launch_dim<128, false>(a, s);
    default: return stream ? launch_dim<256, true>(a, s) : launch_dim<256, false>(a, s);
  }
}

}  // namespace w12
