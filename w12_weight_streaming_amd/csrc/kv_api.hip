// extern "C" entry points of the KV cache, its attention and the sampled tree
// acceptance (declared in include/w12.h). As in w12_api.hip, every call
// checks its arguments on the host and returns before anything is launched
// when one is wrong; nothing here allocates memory.
#include "../../include/w12.h"
#include "kv_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool apart(const void* p, size_t np, const void* q, size_t nq) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a + np <= b || b + nq <= a;
}
w12_status st(hipError_t e) { return e == hipSuccess ? W12_OK : W12_EHIP; }

// Sizes of a cache that the kernels' indexing holds for.
bool cache_ok(const w12_kv_cache* c) {
  if (!c || (c->kvtype != W12_KV_E4M3 && c->kvtype != W12_KV_INT8)) return false;
  if (c->layers < 1 || c->layers > 1024 || c->num_pages < 1 || c->slots < 1 || c->slots > (1 << 20)) return false;
  if (c->kv_heads < 1 || c->kv_heads > w12::kMaxHeads) return false;
  if (c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 96 && c->page_tokens != 128) return false;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return false;
  if (c->recent_rows < c->page_tokens || c->recent_rows % 32 != 0 || c->recent_rows > 1024) return false;
  if (c->max_pages < 1 || (int64_t)c->max_pages * c->page_tokens > (int64_t(1) << 30)) return false;
  if (!c->pages || !c->scales || !c->recent || !c->page_table || !c->len) return false;
  return aligned(c->pages, 16) && aligned(c->scales, 8) && aligned(c->recent, 16) && aligned(c->page_table, 4) &&
         aligned(c->len, 4);
}

w12::KvArgs args_of(const w12_kv_cache* c) {
  w12::KvArgs a{};
  a.pages = c->pages;
  a.scales = c->scales;
  a.recent = c->recent;
  a.table = c->page_table;
  a.len = c->len;
  a.kind = c->kvtype;
  a.layers = c->layers;
  a.num_pages = c->num_pages;
  a.kv_heads = c->kv_heads;
  a.page = c->page_tokens;
  a.dim = c->head_dim;
  a.slots = c->slots;
  a.recent_rows = c->recent_rows;
  a.max_pages = c->max_pages;
  return a;
}

bool step_ok(int32_t num_seq, const int32_t* row_off, int32_t total_rows) {
  return num_seq >= 1 && num_seq <= w12::kStepRows && total_rows >= 1 && total_rows <= w12::kStepRows && row_off;
}
bool heads_ok(const w12_kv_cache* c, int32_t q_heads) {
  return q_heads >= 1 && q_heads <= w12::kMaxHeads && q_heads % c->kv_heads == 0;
}

}  // namespace

extern "C" {

w12_status w12_kv_append(const w12_kv_cache* cache, int32_t layer, int32_t num_seq, const int32_t* slot,
                         const int32_t* row_off, int32_t total_rows, const int32_t* parent, const void* qkv,
                         int qkv_type, int32_t q_heads, const float* rope, int32_t positions, int32_t rot_dim,
                         int32_t interleaved, uint16_t* q, hipStream_t stream) {
  if (!cache_ok(cache) || layer < 0 || layer >= cache->layers || !step_ok(num_seq, row_off, total_rows) ||
      !heads_ok(cache, q_heads))
    return W12_EINVAL;
  if (!qkv || !q || !rope || (qkv_type != W12_Y_F32 && qkv_type != W12_Y_BF16)) return W12_EINVAL;
  if (positions < 1 || rot_dim < 2 || rot_dim > cache->head_dim || rot_dim % 2 != 0) return W12_EINVAL;
  if (!aligned(qkv, 16) || !aligned(q, 16) || !aligned(rope, 4)) return W12_EINVAL;
  const size_t heads = (size_t)total_rows * cache->head_dim;
  if (!apart(q, heads * q_heads * 2, qkv, heads * (q_heads + 2 * cache->kv_heads) * (qkv_type == W12_Y_F32 ? 4 : 2)))
    return W12_EINVAL;
  w12::AppendArgs a{};
  a.c = args_of(cache);
  a.st = {row_off, slot, parent, num_seq, total_rows};
  a.layer = layer;
  a.qkv = qkv;
  a.qkv_f32 = qkv_type == W12_Y_F32;
  a.rope = rope;
  a.positions = positions;
  a.rot = rot_dim;
  a.interleaved = interleaved != 0;
  a.q_heads = q_heads;
  a.q = q;
  return st(w12::launch_kv_append(a, stream));
}

w12_status w12_kv_attention_workspace(const w12_kv_cache* cache, int32_t num_seq, int32_t total_rows, int32_t q_heads,
                                      size_t* bytes) {
  if (!bytes || !cache_ok(cache) || !heads_ok(cache, q_heads) || num_seq < 1 || num_seq > w12::kStepRows ||
      total_rows < 1 || total_rows > w12::kStepRows)
    return W12_EINVAL;
  const int cu = w12::device_cu_count();
  if (cu <= 0) return W12_EHIP;
  *bytes = w12::plan_kv_attention(args_of(cache), cu).ws_bytes;
  return W12_OK;
}

w12_status w12_kv_attention(const w12_kv_cache* cache, int32_t layer, int32_t num_seq, const int32_t* slot,
                            const int32_t* row_off, int32_t total_rows, const int32_t* parent, const uint16_t* q,
                            int32_t q_heads, float scale, uint16_t* out, void* ws, size_t ws_bytes,
                            hipStream_t stream) {
  if (!cache_ok(cache) || layer < 0 || layer >= cache->layers || !step_ok(num_seq, row_off, total_rows) ||
      !heads_ok(cache, q_heads))
    return W12_EINVAL;
  if (!q || !out || !ws || !(scale > 0.0f && scale < __builtin_huge_valf())) return W12_EINVAL;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(ws, 256)) return W12_EINVAL;
  const size_t bytes = (size_t)total_rows * q_heads * cache->head_dim * 2;
  if (!apart(q, bytes, out, bytes)) return W12_EINVAL;
  const int cu = w12::device_cu_count();
  if (cu <= 0) return W12_EHIP;
  w12::AttentionArgs a{};
  a.c = args_of(cache);
  const w12::AttentionPlan p = w12::plan_kv_attention(a.c, cu);
  if (ws_bytes < p.ws_bytes) return W12_ENOSPC;
  if (!apart(ws, p.ws_bytes, out, bytes) || !apart(ws, p.ws_bytes, q, bytes)) return W12_EINVAL;
  a.st = {row_off, slot, parent, num_seq, total_rows};
  a.layer = layer;
  a.q = q;
  a.q_heads = q_heads;
  a.scale = scale;
  a.out = out;
  char* base = static_cast<char*>(ws);
  a.items = base;
  a.part = reinterpret_cast<float*>(base + p.off_part);
  a.part_ml = reinterpret_cast<float*>(base + p.off_ml);
  a.G = p.G;
  return st(w12::launch_kv_attention(a, stream));
}

w12_status w12_kv_commit(const w12_kv_cache* cache, int32_t num_seq, const int32_t* slot, const int32_t* row_off,
                         int32_t total_rows, const int32_t* accept_len, const int32_t* path, int32_t* len_out,
                         hipStream_t stream) {
  if (!cache_ok(cache) || !step_ok(num_seq, row_off, total_rows) || !accept_len || !len_out) return W12_EINVAL;
  w12::CommitArgs a{};
  a.c = args_of(cache);
  a.st = {row_off, slot, nullptr, num_seq, total_rows};
  a.accept_len = accept_len;
  a.path = path;
  a.len_out = len_out;
  return st(w12::launch_kv_commit(a, stream));
}

namespace {
bool sampled_ok(int32_t num_trees, int32_t total_nodes, int32_t vocab) {
  return num_trees >= 1 && total_nodes >= 1 && total_nodes <= 65535 && num_trees <= 65535 && vocab >= 1 &&
         vocab <= (1 << 28);
}
}  // namespace

w12_status tree_accept_sampled_workspace(int32_t num_trees, int32_t total_nodes, int32_t vocab, size_t* bytes) {
  if (!bytes || !sampled_ok(num_trees, total_nodes, vocab)) return W12_EINVAL;
  *bytes = w12::tree_sampled_ws_bytes(num_trees, total_nodes, vocab);
  return W12_OK;
}

w12_status tree_accept_sampled(int32_t num_trees, const int32_t* node_off, int32_t total_nodes, const int32_t* parent,
                               const int32_t* token, const void* logits, int logits_type, int32_t vocab,
                               const float* temperature, const float* draft, const float* u_accept,
                               const float* u_bonus, int32_t* accept_len, int32_t* path, int32_t* bonus, void* ws,
                               size_t ws_bytes, hipStream_t stream) {
  if (!sampled_ok(num_trees, total_nodes, vocab)) return W12_EINVAL;
  if (!node_off || !parent || !token || !logits || !u_accept || !u_bonus || !accept_len || !path || !bonus || !ws)
    return W12_EINVAL;
  if (logits_type != W12_Y_F32 && logits_type != W12_Y_BF16) return W12_EINVAL;
  if (!aligned(ws, 16) || !aligned(logits, logits_type == W12_Y_F32 ? 4 : 2) || !aligned(draft, 4)) return W12_EINVAL;
  if (ws_bytes < w12::tree_sampled_ws_bytes(num_trees, total_nodes, vocab)) return W12_ENOSPC;
  w12::SampledArgs a{};
  a.num_trees = num_trees;
  a.total = total_nodes;
  a.vocab = vocab;
  a.node_off = node_off;
  a.parent = parent;
  a.token = token;
  a.logits = logits;
  a.logits_f32 = logits_type == W12_Y_F32;
  a.temperature = temperature;
  a.draft = draft;
  a.u_accept = u_accept;
  a.u_bonus = u_bonus;
  a.accept_len = accept_len;
  a.path = path;
  a.bonus = bonus;
  a.ws = ws;
  return st(w12::launch_tree_sampled(a, stream));
}

}  // extern "C"
