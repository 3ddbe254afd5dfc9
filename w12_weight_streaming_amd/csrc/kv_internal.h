// Host-side launch interface of the KV-cache kernels (kv_cache.hip,
// kv_attention.hip) and the sampled tree acceptance (tree_sampled.hip), and
// the device helpers they share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w12 {

constexpr int kStepRows = 512;  // rows (and so sequences) of one step, as in w12_gemm
constexpr int kMaxHeads = 256;  // query heads
constexpr int kGroup = 32;      // tokens per fragment group

// The cache's arrays (w12.h) with every size in elements.
struct KvArgs {
  uint8_t* pages;
  float* scales;
  uint16_t* recent;
  const int32_t* table;
  int32_t* len;
  int kind;  // 0 e4m3, 1 int8
  int layers, num_pages, kv_heads, page, dim, slots, recent_rows, max_pages;
};

// The rows of one step: sequence s owns rows [row_off[s], row_off[s + 1]).
struct StepArgs {
  const int32_t* row_off;
  const int32_t* slot;    // null: sequence s uses slot s
  const int32_t* parent;  // null: row i follows row i - 1
  int num_seq, total;
};

struct AppendArgs {
  KvArgs c;
  StepArgs st;
  int layer;
  const void* qkv;
  int qkv_f32;
  const float* rope;
  int positions, rot, interleaved;
  int q_heads;
  uint16_t* q;
};

struct AttentionArgs {
  KvArgs c;
  StepArgs st;
  int layer;
  const uint16_t* q;
  int q_heads;
  float scale;
  uint16_t* out;
  void* items;     // [G] the item each workgroup begins and others go on with
  float* part;     // [2 G][rows of a block][dim] partial sums, not normalised
  float* part_ml;  // [2 G][rows of a block][2] their running maxima and sums
  int G;           // workgroups
  int most_tiles;  // of 32 query rows in a block
};

struct CommitArgs {
  KvArgs c;
  StepArgs st;
  const int32_t* accept_len;
  const int32_t* path;  // null: the first accept_len + 1 rows
  int32_t* len_out;     // [slots]
};

struct SampledArgs {
  int num_trees, total, vocab;
  const int32_t* node_off;
  const int32_t* parent;
  const int32_t* token;
  const void* logits;
  int logits_f32;
  const float* temperature;  // null: 1
  const float* draft;        // null: drafted tokens are certain
  const float* u_accept;
  const float* u_bonus;
  int32_t* accept_len;
  int32_t* path;
  int32_t* bonus;
  void* ws;
};

int device_cu_count();  // of the current device; -1 on failure

hipError_t launch_kv_append(const AppendArgs& a, hipStream_t s);
hipError_t launch_kv_commit(const CommitArgs& a, hipStream_t s);

struct AttentionPlan {
  int G;
  size_t off_part, off_ml, ws_bytes;
};
AttentionPlan plan_kv_attention(const KvArgs& c, int num_cu);
hipError_t launch_kv_attention(const AttentionArgs& a, hipStream_t s);

size_t tree_sampled_ws_bytes(int num_trees, int total, int vocab);
hipError_t launch_tree_sampled(const SampledArgs& a, hipStream_t s);

#ifdef __HIPCC__
// Places (in elements) of a row's dims in the fragment order that pages and
// recent rows share: keys of 32 tokens x 32 dims are [2 halves of 16
// dims][32 tokens][16 dims], values [2 halves][32 dims][16 tokens], half h of
// the values holding tokens 8 i + 4 h + j (j < 4) at i * 4 + j. A fragment is
// one matrix operand for 64 lanes, 16 values each.
__host__ __device__ __forceinline__ int key_at(int t, int d, int dim) {
  return (((t >> 5) * (dim >> 5) + (d >> 5)) * 64 + ((d >> 4) & 1) * 32 + (t & 31)) * 16 + (d & 15);
}
__host__ __device__ __forceinline__ int value_at(int t, int d, int dim) {
  return (((t >> 5) * (dim >> 5) + (d >> 5)) * 64 + ((t >> 2) & 1) * 32 + (d & 31)) * 16 + ((t >> 3) & 3) * 4 + (t & 3);
}

__device__ __forceinline__ size_t page_at(const KvArgs& c, int layer, int page, int head, int v) {
  return ((((size_t)layer * c.num_pages + page) * c.kv_heads + head) * 2 + v) * ((size_t)c.page * c.dim);
}
__device__ __forceinline__ size_t scale_at(const KvArgs& c, int layer, int page, int head, int v) {
  return (((size_t)layer * c.num_pages + page) * c.kv_heads + head) * 2 + v;
}
__device__ __forceinline__ size_t recent_at(const KvArgs& c, int layer, int slot, int head, int v) {
  return ((((size_t)layer * c.slots + slot) * c.kv_heads + head) * 2 + v) * ((size_t)c.recent_rows * c.dim);
}

// Sequence s of a step as every kernel reads it. ok is false where the
// offsets, the slot or the committed length are outside their arrays.
struct SeqView {
  int row0, rows, slot, len, full, tail;
  bool ok;
};
__device__ __forceinline__ SeqView seq_view(const KvArgs& c, const StepArgs& st, int s) {
  SeqView v;
  const int b0 = st.row_off[s], b1 = st.row_off[s + 1];
  v.ok = b0 >= 0 && b0 <= b1 && b1 <= st.total;
  v.row0 = v.ok ? b0 : 0;
  v.rows = v.ok ? b1 - b0 : 0;
  v.slot = st.slot ? st.slot[s] : s;
  if (v.slot < 0 || v.slot >= c.slots) {
    v.ok = false;
    v.slot = 0;
  }
  v.len = c.len[v.slot];
  if (v.len < 0 || v.len > c.max_pages * (long long)c.page) {
    v.ok = false;
    v.len = 0;
  }
  v.full = v.len / c.page;
  v.tail = v.len - v.full * c.page;
  if (v.tail + v.rows > c.recent_rows) v.ok = false;
  return v;
}
// Rows [row0, row0 + rows) meet those of sequence j (where offsets run
// backwards): the later of the two has no rows then, as one whose range is none.
__device__ __forceinline__ bool rows_meet(const int32_t* off, int total, int j, int row0, int rows) {
  const int b0 = off[j], b1 = off[j + 1];
  return b0 >= 0 && b1 <= total && b0 < b1 && b0 < row0 + rows && b1 > row0;
}
#endif

}  // namespace w12
