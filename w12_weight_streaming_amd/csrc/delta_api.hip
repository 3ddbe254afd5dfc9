// extern "C" entry points of the recurrent layers and of the norms (declared
// in include/w12.h). Every call checks its arguments on the host and returns
// before anything is launched when one is wrong; nothing here allocates memory.
#include <initializer_list>

#include "../../include/w12.h"
#include "delta_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool apart(const void* p, size_t np, const void* q, size_t nq) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a + np <= b || b + nq <= a;
}
bool finite(float x) { return x - x == 0.0f; }
bool ydtype(int t) { return t == W12_Y_F32 || t == W12_Y_BF16; }
size_t bytes_of(int t) { return t == W12_Y_F32 ? 4 : 2; }
w12_status st(hipError_t e) { return e == hipSuccess ? W12_OK : W12_EHIP; }

// Sizes that the kernels' indexing holds for.
bool cache_ok(const w12_delta_cache* c) {
  if (!c || c->layers < 1 || c->layers > 1024 || c->slots < 1 || c->slots > (1 << 20)) return false;
  if (c->step_rows < 1 || c->step_rows > 65536) return false;
  if (c->key_heads < 1 || c->value_heads < 1 || c->value_heads > w12::kMaxHeads || c->value_heads % c->key_heads != 0)
    return false;
  if (c->key_dim != 64 && c->key_dim != 128) return false;
  if (c->value_dim != 64 && c->value_dim != 128) return false;
  if (c->conv_width < 2 || c->conv_width > 4) return false;
  if (!c->state || !c->conv || !c->raw || !c->kv || !c->gates || !c->delta) return false;
  return aligned(c->state, 16) && aligned(c->conv, 16) && aligned(c->raw, 16) && aligned(c->kv, 16) &&
         aligned(c->gates, 16) && aligned(c->delta, 16);
}

w12::DeltaArgs args_of(const w12_delta_cache* c) {
  w12::DeltaArgs a{};
  a.state = c->state;
  a.conv = c->conv;
  a.raw = c->raw;
  a.kv = c->kv;
  a.gates = c->gates;
  a.delta = c->delta;
  a.layers = c->layers;
  a.slots = c->slots;
  a.step_rows = c->step_rows;
  a.key_heads = c->key_heads;
  a.value_heads = c->value_heads;
  a.key_dim = c->key_dim;
  a.value_dim = c->value_dim;
  a.width = c->conv_width;
  a.kv_width = c->key_heads * c->key_dim + c->value_heads * c->value_dim;
  a.channels = a.kv_width + c->key_heads * c->key_dim;
  return a;
}

bool step_ok(const w12_delta_cache* c, int32_t num_seq, const int32_t* slot, const int32_t* row_off, int32_t total_rows,
             const int32_t* parent) {
  return num_seq >= 1 && num_seq <= w12::kStepRows && total_rows >= 1 && total_rows <= w12::kStepRows &&
         total_rows <= c->step_rows && row_off && aligned(row_off, 4) && aligned(slot, 4) && aligned(parent, 4);
}

// Bytes from the first value of `rows` rows of `values`, `stride` values apart, to behind the last.
size_t span(int64_t rows, int64_t values, int64_t stride, int type) {
  return ((size_t)(rows - 1) * (size_t)stride + (size_t)values) * bytes_of(type);
}

// What a call reads or writes; p null: nothing.
struct Range {
  const void* p;
  size_t bytes;
};
// Nothing that is written lies over what the same call reads.
bool clear(std::initializer_list<Range> written, std::initializer_list<Range> read) {
  for (const Range& w : written)
    for (const Range& r : read)
      if (w.p && r.p && !apart(w.p, w.bytes, r.p, r.bytes)) return false;
  return true;
}
size_t off_bytes(int32_t num_seq) { return ((size_t)num_seq + 1) * 4; }

// `bytes` at p meet none of the cache's arrays.
bool apart_of(const w12::DeltaArgs& a, const void* p, size_t bytes) {
  const size_t steps = (size_t)a.layers * a.step_rows, slots = (size_t)a.layers * a.slots;
  return apart(p, bytes, a.state, slots * a.value_heads * a.key_dim * a.value_dim * 4) &&
         apart(p, bytes, a.conv, slots * (a.width - 1) * a.channels * 2) && apart(p, bytes, a.raw, steps * a.channels * 2) &&
         apart(p, bytes, a.kv, steps * a.kv_width * 2) && apart(p, bytes, a.gates, steps * 2 * a.value_heads * 4) &&
         apart(p, bytes, a.delta, steps * a.value_heads * a.value_dim * 4);
}

}  // namespace

extern "C" {

w12_status w12_delta_append(const w12_delta_cache* cache, int32_t layer, int32_t num_seq, const int32_t* slot,
                            const int32_t* row_off, int32_t total_rows, const int32_t* parent, const void* qkv,
                            int64_t qkv_stride, const void* ba, int64_t ba_stride, int type, const float* conv_weight,
                            const float* conv_bias, const float* a_log, const float* dt_bias, uint16_t* q,
                            hipStream_t stream) {
  if (!cache_ok(cache) || layer < 0 || layer >= cache->layers || !step_ok(cache, num_seq, slot, row_off, total_rows, parent))
    return W12_EINVAL;
  if (!qkv || !ba || !conv_weight || !a_log || !dt_bias || !q || !ydtype(type)) return W12_EINVAL;
  w12::DeltaAppendArgs a{};
  a.c = args_of(cache);
  constexpr int64_t kMost = int64_t(1) << 32;
  if (qkv_stride < a.c.channels || qkv_stride > kMost || ba_stride < 2 * a.c.value_heads || ba_stride > kMost)
    return W12_EINVAL;
  if ((size_t)qkv_stride * bytes_of(type) % 16 != 0 || !aligned(qkv, 16) || !aligned(q, 16) ||
      !aligned(ba, bytes_of(type)) || !aligned(conv_weight, 16) || !aligned(conv_bias, 16) || !aligned(a_log, 4) ||
      !aligned(dt_bias, 4))
    return W12_EINVAL;
  const size_t qb = (size_t)total_rows * a.c.key_heads * a.c.key_dim * 2;
  const size_t wb = (size_t)a.c.channels * 4, hb = (size_t)a.c.value_heads * 4;
  const size_t steps = (size_t)a.c.layers * a.c.step_rows;
  if (!apart_of(a.c, q, qb) ||
      !clear({{q, qb},
              {a.c.raw, steps * a.c.channels * 2},
              {a.c.kv, steps * a.c.kv_width * 2},
              {a.c.gates, steps * 2 * a.c.value_heads * 4}},
             {{qkv, span(total_rows, a.c.channels, qkv_stride, type)},
              {ba, span(total_rows, 2 * a.c.value_heads, ba_stride, type)},
              {conv_weight, wb * a.c.width},
              {conv_bias, wb},
              {a_log, hb},
              {dt_bias, hb},
              {slot, (size_t)num_seq * 4},
              {row_off, off_bytes(num_seq)},
              {parent, (size_t)total_rows * 4}}))
    return W12_EINVAL;
  a.st = {row_off, slot, parent, num_seq, total_rows};
  a.layer = layer;
  a.qkv = qkv;
  a.qkv_stride = qkv_stride;
  a.ba = ba;
  a.ba_stride = ba_stride;
  a.f32 = type == W12_Y_F32;
  a.conv_weight = conv_weight;
  a.conv_bias = conv_bias;
  a.a_log = a_log;
  a.dt_bias = dt_bias;
  a.q = q;
  return st(w12::launch_delta_append(a, stream));
}

w12_status w12_delta_rule(const w12_delta_cache* cache, int32_t layer, int32_t num_seq, const int32_t* slot,
                          const int32_t* row_off, int32_t total_rows, const int32_t* parent, const uint16_t* q,
                          float scale, int32_t keep, uint16_t* out, hipStream_t stream) {
  if (!cache_ok(cache) || layer < 0 || layer >= cache->layers || !step_ok(cache, num_seq, slot, row_off, total_rows, parent))
    return W12_EINVAL;
  if (!q || !out || !finite(scale) || (keep && parent)) return W12_EINVAL;
  if (!aligned(q, 16) || !aligned(out, 16)) return W12_EINVAL;
  w12::DeltaRuleArgs a{};
  a.c = args_of(cache);
  const size_t ob = (size_t)total_rows * a.c.value_heads * a.c.value_dim * 2;
  const size_t vb = (size_t)a.c.value_heads * a.c.value_dim * 4;  // a row's deltas
  const size_t steps = (size_t)a.c.layers * a.c.step_rows, slots = (size_t)a.c.layers * a.c.slots;
  if (!apart_of(a.c, out, ob) || !clear({{out, ob},
                                         {keep ? nullptr : a.c.delta, steps * vb},
                                         {keep ? a.c.state : nullptr, slots * a.c.key_dim * vb},
                                         {keep ? a.c.conv : nullptr, slots * (a.c.width - 1) * a.c.channels * 2}},
                                        {{q, (size_t)total_rows * a.c.key_heads * a.c.key_dim * 2},
                                         {slot, (size_t)num_seq * 4},
                                         {row_off, off_bytes(num_seq)},
                                         {parent, (size_t)total_rows * 4}}))
    return W12_EINVAL;
  a.st = {row_off, slot, parent, num_seq, total_rows};
  a.layer = layer;
  a.q = q;
  a.scale = scale;
  a.keep = keep != 0;
  a.out = out;
  return st(w12::launch_delta_rule(a, stream));
}

w12_status w12_delta_commit(const w12_delta_cache* cache, int32_t num_seq, const int32_t* slot, const int32_t* row_off,
                            int32_t total_rows, const int32_t* accept_len, const int32_t* path, int32_t* kept,
                            hipStream_t stream) {
  if (!cache_ok(cache) || !step_ok(cache, num_seq, slot, row_off, total_rows, nullptr) || !accept_len || !kept ||
      !aligned(accept_len, 4) || !aligned(path, 4) || !aligned(kept, 4))
    return W12_EINVAL;
  w12::DeltaCommitArgs a{};
  a.c = args_of(cache);
  const size_t nb = (size_t)num_seq * 4, slots = (size_t)a.c.layers * a.c.slots;
  if (!apart_of(a.c, kept, nb) ||
      !clear({{kept, nb},
              {a.c.state, slots * a.c.value_heads * a.c.key_dim * a.c.value_dim * 4},
              {a.c.conv, slots * (a.c.width - 1) * a.c.channels * 2}},
             {{accept_len, nb}, {path, (size_t)total_rows * 4}, {slot, nb}, {row_off, off_bytes(num_seq)}}))
    return W12_EINVAL;
  a.st = {row_off, slot, nullptr, num_seq, total_rows};
  a.accept_len = accept_len;
  a.path = path;
  a.kept = kept;
  return st(w12::launch_delta_commit(a, stream));
}

w12_status w12_norm(int64_t rows, int32_t groups, int32_t width, const void* y, int y_type, int64_t y_stride,
                    const float* post_weight, const void* gate, int gate_type, int64_t gate_stride, float scale,
                    void* h, int h_type, const float* weight, float eps, uint16_t* out, hipStream_t stream) {
  if (rows < 1 || rows > (1 << 24) || groups < 1 || groups > 1024 || width < 1 || width > 32768) return W12_EINVAL;
  if (!out || (!y && (!h || gate || post_weight)) || !(eps > 0.0f) || !finite(eps) || !finite(scale)) return W12_EINVAL;
  const int64_t wide = (int64_t)groups * width;
  constexpr int64_t kMost = int64_t(1) << 32;
  if (y && (!ydtype(y_type) || y_stride < wide || y_stride > kMost || !aligned(y, bytes_of(y_type)))) return W12_EINVAL;
  if (gate && (!ydtype(gate_type) || gate_stride < wide || gate_stride > kMost || !aligned(gate, bytes_of(gate_type))))
    return W12_EINVAL;
  if (h && (!ydtype(h_type) || !aligned(h, bytes_of(h_type)))) return W12_EINVAL;
  if (!aligned(out, 2) || !aligned(post_weight, 4) || !aligned(weight, 4)) return W12_EINVAL;
  const size_t ob = (size_t)rows * wide * 2, hb = h ? (size_t)rows * wide * bytes_of(h_type) : 0;
  const size_t yb = y ? span(rows, wide, y_stride, y_type) : 0, gb = gate ? span(rows, wide, gate_stride, gate_type) : 0;
  if ((h && !apart(out, ob, h, hb)) || (y && !apart(out, ob, y, yb)) || (gate && !apart(out, ob, gate, gb)))
    return W12_EINVAL;
  if (h && ((y && !apart(h, hb, y, yb)) || (gate && !apart(h, hb, gate, gb)))) return W12_EINVAL;
  for (const float* w : {post_weight, weight})
    if (w && (!apart(out, ob, w, (size_t)width * 4) || (h && !apart(h, hb, w, (size_t)width * 4)))) return W12_EINVAL;
  w12::NormArgs a{};
  a.rows = rows;
  a.groups = groups;
  a.width = width;
  a.y = y;
  a.y_f32 = y_type == W12_Y_F32;
  a.y_stride = y_stride;
  a.post_weight = post_weight;
  a.gate = gate;
  a.gate_f32 = gate_type == W12_Y_F32;
  a.gate_stride = gate_stride;
  a.scale = scale;
  a.h = h;
  a.h_f32 = h_type == W12_Y_F32;
  a.weight = weight;
  a.eps = eps;
  a.out = out;
  return st(w12::launch_norm(a, stream));
}

}  // extern "C"
