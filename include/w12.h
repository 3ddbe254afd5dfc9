/*
 * w12.h -- C ABI of libw12: lossless 12-bit (W12) weight streaming for the
 * verification pass of greedy speculative decoding, on AMD Instinct MI355X
 * (gfx950).
 *
 * Sources for what each call computes:
 *   [S1] "SpecPilot: Autonomous Algorithm Discovery and Systems Optimization
 *        for Speculative Decoding", long-form summary (jaehun.me):
 *        section 1.1 (greedy acceptance), 1.2 (lossless = exact-pass argmax),
 *        4.1 (W12 format, 12 KB records, deterministic stream-K GEMM, LM
 *        head argmax), 4.3 (tree verification: longest matching path + bonus).
 *   [S2] the same paper's digest page (agihunt.info), W12 paragraph (sign +
 *        4-bit exponent offset + all 7 mantissa bits, load-time check).
 *   [S3] "Speculative decoding" (poot-llm docs), "What a round guarantees"
 *        (greedy rows keep drafts equal to the argmax, then one more token)
 *        and "What is refused" (typed refusal before anything runs).
 *
 * Conventions (all calls):
 *   - Every pointer argument is DEVICE memory owned by the caller, except
 *     `const w12_matrix *` descriptors and `size_t *` / `int64_t` outputs of
 *     the *_workspace queries, which live in host memory.
 *   - Calls are asynchronous on `stream` (a hipStream_t; NULL = the null
 *     stream) and return as soon as the kernels are enqueued.
 *   - Argument errors return W12_EINVAL before anything is launched (null
 *     pointers, shapes the format cannot hold, m outside [1, 512], bf16
 *     matrices / records / x / y not 16-byte aligned, e_top and u32 arrays
 *     not 4-byte aligned); a
 *     workspace smaller than its query returns W12_ENOSPC; a failed launch
 *     returns W12_EHIP.  Errors found on the device (a corrupt packed
 *     weight, an invalid tree) are reported through outputs, as each call
 *     states.  The library never allocates memory.
 *   - Workspaces ("ws") must be zero-filled before their first use. A
 *     workspace holds arrival counters, which every completed call returns
 *     to zero, and partial sums, which a call writes before it reads them;
 *     so one allocation serves any number of calls.  Calls that overlap in
 *     time must not share a workspace.  Where a call says "content ignored"
 *     it leaves any content behind: such a workspace goes to no product or
 *     head afterwards, unless it is zero-filled again.
 *
 * W12 layout (readings of [S1] 4.1 and [S2] for gfx950):
 *   N output channels x K inputs, N % 32 == 0, K % 256 == 0, K <= 2^20.
 *   e_top[n]   window top E_n (biased bf16 exponent) in [16, 254]; the
 *              window [E_n - 15, E_n] is the one holding the most normal
 *              weights of channel n (smallest E_n on ties).
 *   records    N*K*3/2 bytes; record (s, r) = channels [32s, 32s+32) x
 *              k [256r, 256r+256) at byte (s*(K/256) + r) * 12288.  Bytes
 *              [0, 8192) hold the 8-bit view hi8 = s<<7 | o<<3 | m>>4
 *              (o = e - (E_n - 15)), bytes [8192, 12288) the low mantissa
 *              nibbles.  Weight (c, k') of a record, subtile t = k'/32,
 *              half h = (k'%32)/16, j = k'%16, lane = c + 32h:
 *                hi8 at t*1024 + lane*16 + j,
 *                lo4 at 8192 + t*512 + lane*8 + 4*(j/8) + j%4, high nibble
 *                when j%8 < 4, low nibble otherwise.
 *              Escaped weights (zero, denormal, Inf/NaN, out of window) hold
 *              code 0 and are listed in `esc`.
 *   esc_off    [N*K/1024 + 1] u32 offsets into esc, one per escape block
 *              (strip s, record r, subtile t), block id (s*(K/256)+r)*8 + t.
 *   esc        [max(1, esc_off[last])] u32 entries (the array always holds
 *              at least one element) bits<<16 | c<<5 | kk, c the
 *              channel in the strip, kk = k % 32; (c, kk) ascending within a
 *              block, so each channel's list runs in ascending k.
 */
#ifndef W12_H
#define W12_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  W12_OK = 0,
  W12_EINVAL = -1,  /* bad argument; nothing launched                    */
  W12_ENOSPC = -2,  /* workspace smaller than the matching query         */
  W12_EHIP = -3,    /* a HIP runtime call or kernel launch failed        */
  W12_ECORRUPT = -4 /* the load-time check found weights that do not
                       restore bit-for-bit: the weights are refused
                       ([S1] 4.1, [S2]; [S3] "What is refused"). No call
                       of the library returns it: w12_check reports a
                       count through device memory, and the caller that
                       reads a non-zero count refuses the weights with
                       this status (the Python binding raises it).     */
} w12_status;

typedef enum { W12_Y_F32 = 0, W12_Y_BF16 = 1 } w12_ydtype;

/* Device-resident W12 matrix (the five buffers above). */
typedef struct w12_matrix {
  int64_t n, k;
  const uint8_t *records;
  const uint8_t *e_top;
  const uint32_t *esc_off;
  const uint32_t *esc;
} w12_matrix;

/* Human-readable name of a w12_status (static string). */
const char *w12_strerror(int status);

/* ABI version, bumped on any layout or signature change. */
int w12_abi_version(void);

/* Number of escape blocks N*K/1024; esc_off holds one more entry. */
int64_t w12_num_blocks(int64_t n, int64_t k);

/*
 * w12_pack_plan -- first half of packing ([S1] 4.1: the weights are
 * converted once, at load; per output channel the 16-binade exponent window
 * holding the most weights, everything outside it on the escape list;
 * [S2] W12 paragraph).
 *   w        [n, k] bf16 bit patterns, row-major (read only).
 *   e_top    [n] out: window tops E_n.
 *   esc_off  [w12_num_blocks(n,k) + 1] out: escape offsets; esc_off[last]
 *            is the escape count the caller reads to size `esc`.
 */
w12_status w12_pack_plan(const uint16_t *w, int64_t n, int64_t k,
                         uint8_t *e_top, uint32_t *esc_off, hipStream_t stream);

/*
 * w12_pack -- second half of packing ([S1] 4.1; [S2]): writes the 12 KB
 * records (8-bit view plane, then low-nibble plane) and the escape entries
 * (exact bf16 bits of every weight outside its channel's window).
 *   e_top, esc_off  from w12_pack_plan on the same w.
 *   records         [n*k*3/2] out.
 *   esc             [esc_capacity] out; entries past esc_capacity are
 *                   dropped (the load-time check then fails), so pass
 *                   esc_capacity >= esc_off[last].
 */
w12_status w12_pack(const uint16_t *w, int64_t n, int64_t k,
                    const uint8_t *e_top, const uint32_t *esc_off,
                    uint8_t *records, uint32_t *esc, int64_t esc_capacity,
                    hipStream_t stream);

/* w12_decode -- restore the bf16 weights [n, k] (row-major) exactly
 * ([S1] 4.1: escapes restored exactly; the same in-register decode the GEMM
 * uses). */
w12_status w12_decode(const w12_matrix *w, uint16_t *out, hipStream_t stream);

/* w12_check -- load-time bit-for-bit check ([S1] 4.1, [S2]): decodes every
 * weight and ADDS the number that differ from ref [n, k] to *mismatches
 * (device u64; the caller zeroes it). Non-zero means refuse the weights
 * (W12_ECORRUPT). An escape block whose offsets are inconsistent
 * (esc_off[b+1] < esc_off[b], esc_off[b+1] > esc_off[last], or more than
 * the block's 1024 weights) counts all of its 1024 weights as mismatches and
 * reads no entry. Reads of esc stay below esc_off[last], which the caller
 * vouches for as the length of esc. w12_decode applies the same bounds; its
 * output for such a block is the records' codes without escapes. */
w12_status w12_check(const w12_matrix *w, const uint16_t *ref,
                     unsigned long long *mismatches, hipStream_t stream);

/* Workspace bytes w12_gemm needs for this shape (host output). The
 * workspace holds what the deterministic split of the k reduction needs
 * ([S1] 4.1: stream-K with a fixed summation order): one arrival counter per
 * output tile, the partial sums of the tiles split between workgroups, the
 * argmax keys of the head, and x rearranged into matrix-core fragments. The
 * size depends on the device's compute-unit count, which the library reads
 * once per device id and keeps for the life of the process (the only state
 * the library holds besides the no-allocation entry point's scratch). */
w12_status w12_gemm_workspace(int64_t n, int64_t k, int64_t m, size_t *bytes);

/*
 * w12_gemm -- verify GEMM ([S1] 4.1): y[i, c] = sum_k x[i, k] * W[c, k] for
 * the m verify rows, streaming every W12 record from HBM once, restoring it
 * in registers, fp32 accumulation. Rows m <= 4 use a VALU dot-product path,
 * m >= 5 bf16 MFMA (more than 192 rows run as several launches of at most
 * 192 rows, each streaming W again). The reduction over k is split across workgroups in a
 * fixed order (stream-K), so results are bitwise reproducible.
 *   x   [m, k] bf16 row-major, 1 <= m <= 512.
 *   y   [m, n] row-major, fp32 (W12_Y_F32) or bf16 (W12_Y_BF16, the
 *       round-to-nearest-even of the same fp32 result).
 *   ws  zero-filled workspace of >= w12_gemm_workspace bytes.
 */
w12_status w12_gemm(const w12_matrix *w, const uint16_t *x, int64_t m,
                    void *y, int ytype, void *ws, size_t ws_bytes,
                    hipStream_t stream);

/*
 * w12_gemm_noalloc -- w12_gemm for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc): the same kernels and results, bit for bit, with the
 * workspace taken from a static device array of the library
 * (W12_NOALLOC_SCRATCH_BYTES per device, reserved when the library is
 * loaded and held until the process ends). The call allocates nothing.
 *   Arguments and layouts as w12_gemm, without ws / ws_bytes.
 *   Returns W12_ENOSPC, before launching anything, when w12_gemm_workspace
 *   for the shape exceeds W12_NOALLOC_SCRATCH_BYTES. At 256 compute units
 *   every m <= 512 fits for k <= 400000 (192-row launches need 51.6 MB;
 *   5 <= m <= 64 adds 128 * k bytes of x fragments).
 *   The first call on a device looks up the array's device address and
 *   enqueues one kernel on `stream` that zero-fills it; every completed call
 *   leaves its counters at zero again.
 *   All calls on one device share that device's array: calls that overlap in
 *   time on one device (other streams, other threads) race and give wrong
 *   results. Serialise them.
 */
#define W12_NOALLOC_SCRATCH_BYTES (64u << 20)
w12_status w12_gemm_noalloc(const w12_matrix *w, const uint16_t *x, int64_t m,
                            void *y, int ytype, hipStream_t stream);

/* Workspace bytes w12_head_argmax needs (host output). */
w12_status w12_head_argmax_workspace(int64_t n, int64_t k, int64_t m, size_t *bytes);

/*
 * w12_head_argmax -- LM head + greedy token ([S1] 1.1, 4.1): for each verify
 * row i, idx[i] = the lowest vocabulary id v attaining max_v logits[i, v],
 * logits = x W^T computed as in w12_gemm (never written to memory).
 *   idx     [m] int32 out; maxval [m] fp32 out (may be NULL).
 */
w12_status w12_head_argmax(const w12_matrix *head, const uint16_t *x, int64_t m,
                           int32_t *idx, float *maxval, void *ws, size_t ws_bytes,
                           hipStream_t stream);

/*
 * Certified INT8 LM head ([S1] 4.1, the LM-head paragraph: an INT8 copy of
 * the head, a per-row Cauchy-Schwarz error bound that proves which tokens
 * cannot be the argmax, exact rescoring of the survivors only; the argmax
 * does not change).
 *
 * The INT8 copy of an n x k head (device memory, caller-owned):
 *   q       [n*k] int8: per vocabulary row and block of 32 consecutive k,
 *           every weight the W12 pack keeps in its window is
 *           q = RNE(w / 2^s), s the smallest integer with all of the
 *           block's window weights |w| <= 127 * 2^s; weights W12 escapes
 *           are 0 (they come back exactly from the W12 head's escape
 *           list). Layout: 8 KB records, record (strip, r) at
 *           (strip*(k/256) + r) * 8192, weight (c, k') at the byte W12's
 *           8-bit view uses: t*1024 + (c + 32h)*16 + j.
 *   qexp    [n*k/32] u8 block codes s + 133 (0: no window weight in the
 *           block) at ((strip*(k/256) + r)*8 + t)*32 + c.
 *   cbound  [n] fp32 per-row constant ||e|| + 2 k 2^-24 ||w'||, rounded up
 *           (w' = the copy's weights with the escapes exact, e = w - w').
 */
typedef struct w12_cert8 {
  int64_t n, k;
  const int8_t *q;
  const uint8_t *qexp;
  const float *cbound;
} w12_cert8;

/* w12_cert8_pack -- build the INT8 copy from the bf16 head w [n, k] and the
 * window tops e_top [n] that w12_pack_plan gave for the same w (load time).
 * q, qexp, cbound as above (q 16-byte aligned, cbound 4-byte aligned). */
w12_status w12_cert8_pack(const uint16_t *w, int64_t n, int64_t k, const uint8_t *e_top,
                          int8_t *q, uint8_t *qexp, float *cbound, hipStream_t stream);

/* Workspace bytes w12_head_argmax_certified needs (host output). */
w12_status w12_head_argmax_certified_workspace(int64_t n, int64_t k, int64_t m, size_t *bytes);

/*
 * w12_head_argmax_certified -- the certified head argmax for 1 <= m <= 64
 * rows: an MFMA pass over the INT8 copy gives A = x.w' (fp32) per row and
 * vocabulary row, with bounds A +- B, B = ||x|| cbound + 1e-6 (rounded
 * outward); LB = the row's largest lower bound; every group of 4 vocabulary
 * rows whose upper bound reaches LB is rescored exactly from the W12 head
 * (its records and escapes, fp32 accumulation). idx[i] = the lowest id
 * attaining the largest rescored logit, which is the exact head argmax
 * (within the same floating-point allowance as w12_head_argmax).
 *   head    the W12 head of the same weights; cert its INT8 copy (same n, k).
 *   idx     [m] int32 out; maxval [m] fp32 out or NULL (the winning logit);
 *   rescored [m] int32 out or NULL: vocabulary rows rescored per row.
 *   ws      zero-filled workspace of >= w12_head_argmax_certified_workspace
 *           bytes; every completed call leaves its counters and keys at
 *           zero again, so one workspace serves certified calls of any
 *           shape (but not w12_gemm / w12_head_argmax calls: their
 *           counters sit at other offsets).
 * Errors: W12_EINVAL also when one workgroup's share of the head spans more
 * than 4096 vocabulary rows (n above about 900000 at 256 compute units).
 */
w12_status w12_head_argmax_certified(const w12_matrix *head, const w12_cert8 *cert, const uint16_t *x,
                                     int64_t m, int32_t *idx, float *maxval, int32_t *rescored,
                                     void *ws, size_t ws_bytes, hipStream_t stream);

/*
 * w12_gemm_qpass, w12_head_argmax_qpass -- the Q pass ([S1] 4.3): the same
 * products read from the 8-bit view alone (the first 2/3 of every record),
 * every dropped low mantissa nibble taken at its midpoint 0b1000; escaped
 * weights are restored from the escape list as in the exact pass. Arguments,
 * layouts, workspace (w12_gemm_workspace) and errors as w12_gemm and
 * w12_head_argmax; results are bitwise reproducible but are not those of the
 * exact pass.
 */
w12_status w12_gemm_qpass(const w12_matrix *w, const uint16_t *x, int64_t m,
                          void *y, int ytype, void *ws, size_t ws_bytes,
                          hipStream_t stream);
w12_status w12_head_argmax_qpass(const w12_matrix *head, const uint16_t *x, int64_t m,
                                 int32_t *idx, float *maxval, void *ws, size_t ws_bytes,
                                 hipStream_t stream);

/*
 * w12_tree_build -- best-first draft trees under one shared row budget
 * ([S1] 4.2: every edge scored by the log-softmax of the child given its
 * parent, the nodes of highest path score kept; [S1] 4.4: one node budget
 * shared by all requests of a step, filled from the highest path score down,
 * each request's share a prefix-closed tree).
 *   num_req R in [1, 128]; positions D in [1, 16]; k K in [1, 16].
 *   lp    [R][D][K][K] fp32: lp[r][d][i][j] = edge score from candidate i of
 *         position d - 1 (the root for d = 0, row i = 0) to candidate j of
 *         position d; expected <= 0 (a log-softmax over j), finite.
 *   tok   [R][D][K] int32 candidate tokens; depth [R] int32 positions drafted
 *         per request (values outside [0, D] are clamped); root [R] int32
 *         committed token of each request.
 *   budget rows in all, roots included: R <= budget, budget - R <= 1023 and
 *         R * (budget - R) <= 8192.
 * Order: path score (the binary32 sum of edge scores, accumulated from the
 * root in path order) highest first, then depth, then request index, then the
 * path of child ranks (a parent's children ranked by edge score, equal scores
 * by candidate index).
 * Output (device memory, caller-owned, the layout tree_accept reads):
 *   node_off [R+1]; then per request its root row (parent -1, token root[r],
 *   depth 0, score 0) followed by its draft nodes in that order, parent local
 *   to the request; parent, token, node_depth, score hold node_off[R] rows
 *   (at most budget; fewer when the lattices run out of nodes). node_depth and
 *   score may be NULL.
 * Workspace: w12_tree_build_workspace bytes, 16-byte aligned, content ignored.
 * Errors: W12_EINVAL for shapes or pointers outside the above, W12_ENOSPC for
 * a small workspace, W12_EHIP for a launch error.
 */
w12_status w12_tree_build_workspace(int32_t num_req, int32_t budget, size_t *bytes);
w12_status w12_tree_build(int32_t num_req, int32_t positions, int32_t k, const float *lp,
                          const int32_t *tok, const int32_t *depth, const int32_t *root,
                          int32_t budget, void *ws, size_t ws_bytes, int32_t *node_off,
                          int32_t *parent, int32_t *token, int32_t *node_depth, float *score,
                          hipStream_t stream);

/*
 * tree_accept -- greedy tree verification ([S1] 1.1, 4.3; [S3]).
 * Trees are concatenated: tree t owns nodes [node_off[t], node_off[t+1]),
 * node_off[0] = 0, node_off[num_trees] = total_nodes; node i of a tree is
 * verify row node_off[t] + i, with tree-local parent[i] (-1 for the root,
 * else in [0, i)), draft token token[i] and the target's argmax[i] for that
 * row. A node is accepted when every edge on its root path satisfies
 * token[child] == argmax[parent]. Per tree:
 *   accept_len[t] = depth of the deepest accepted node (lowest index on
 *                   ties) = number of accepted drafts (tau = accept_len+1);
 *   path[node_off[t] + j] = tree-local node at depth j of that path for
 *                   j <= accept_len, -1 after it;
 *   bonus[t]      = argmax of the deepest accepted node's row.
 * A tree with no nodes, a root parent other than -1, a parent outside
 * [0, i), or offsets outside [0, total_nodes] gets accept_len = bonus = -1
 * and an all -1 path (device-detected; the call itself returns W12_OK).
 * total_nodes (the length of parent, token, argmax and path) is what the
 * kernel checks device-side offsets against, so that a corrupt node_off
 * never reads or writes past those arrays.
 */
w12_status tree_accept(int32_t num_trees, const int32_t *node_off,
                       int32_t total_nodes, const int32_t *parent,
                       const int32_t *token, const int32_t *argmax,
                       int32_t *accept_len, int32_t *path, int32_t *bonus,
                       hipStream_t stream);

/*
 * KV cache of the verify pass. [S1] 4.3: a pass runs the target over draft
 * trees and keeps one root path of each; [S1] 4.4: prompts share the pass,
 * their rows a chain. The cache holds, per layer:
 *   pages   [layers][num_pages][kv_heads][2 (K, V)][page_tokens * head_dim]
 *           8-bit codes of whole blocks of page_tokens committed tokens,
 *           W12_KV_E4M3 (OCP e4m3) or W12_KV_INT8;
 *   scales  [layers][num_pages][kv_heads][2] fp32: a code stands for
 *           code * scale, one scale per block, head and K or V, at least
 *           2^-90 (or NaN: the block reads as NaN);
 *   recent  [layers][slots][kv_heads][2][recent_rows * head_dim] bf16: the
 *           committed tokens of a sequence's unfinished block (its first
 *           len % page_tokens rows), then the rows of the current step.
 * and for all layers:
 *   page_table [slots][max_pages] int32: page of each block of a sequence;
 *   len        [slots] int32: committed tokens of each sequence.
 * A block is quantised once, when its last token is committed, from bf16: the
 * pages depend on the accepted tokens only, not on rejected drafts or on how
 * tokens were grouped into steps.
 * Order inside a block and inside the recent rows: keys of 32 tokens x 32
 * dims lie as [2 halves of 16 dims][32 tokens][16 dims], values as [2][32
 * dims][16 tokens], half h holding tokens 8 i + 4 h + j (i, j < 4) at 4 i + j;
 * such fragments are ordered by 32 tokens, then by 32 dims.
 * Sizes: page_tokens 32, 64, 96 or 128; head_dim 64, 128 or 256; recent_rows
 * a multiple of 32 in [page_tokens, 1024]; kv_heads <= 256; slots <= 2^20;
 * max_pages * page_tokens <= 2^30; layers <= 1024; query heads a multiple of
 * kv_heads, at most 256. pages and recent 16-byte, scales 8-byte aligned.
 *
 * A step's calls share its rows: sequence s owns rows [row_off[s],
 * row_off[s + 1]) of total_rows (at most 512, at most 512 sequences), a tree
 * with tree-local parents as in tree_accept, or, with parent NULL, a chain
 * (row i follows row i - 1: prompts, plain decoding, chains of drafts). slot
 * [num_seq] names each sequence's slot (NULL: its own index). row_off
 * ascends; a sequence whose range runs backwards, leaves [0, total_rows) or
 * meets an earlier sequence's has no rows. Rows of no sequence are left as
 * they are.
 */
typedef enum { W12_KV_E4M3 = 0, W12_KV_INT8 = 1 } w12_kvtype;

typedef struct w12_kv_cache {
  int32_t kvtype, layers, num_pages, kv_heads, page_tokens, head_dim, slots, recent_rows, max_pages;
  uint8_t *pages;
  float *scales;
  uint16_t *recent;
  const int32_t *page_table;
  int32_t *len;
} w12_kv_cache;

/*
 * w12_kv_append -- rotates a step's queries and keys by their positions and
 * puts keys and values behind the sequence's committed tokens, as rows that
 * w12_kv_attention sees and w12_kv_commit keeps or drops. len is not changed:
 * appending again overwrites the step's rows.
 *   qkv  [total_rows][(q_heads + 2 kv_heads) * head_dim] fp32 or bf16
 *        (qkv_type a w12_ydtype): query heads, key heads, value heads, as the
 *        fused Wq|Wk|Wv product writes them.
 *   rope [positions][rot_dim] fp32: cosines of the rot_dim / 2 angles of a
 *        position, then their sines. The row at depth d of its tree has
 *        position len + d. The first rot_dim dims (even) of each query and
 *        key head turn in pairs (i, i + rot_dim / 2), or (2 i, 2 i + 1) if
 *        interleaved; computed in fp32, rounded to bf16 once.
 *   q    [total_rows][q_heads][head_dim] bf16 out: the rotated queries; not qkv's memory.
 * Device-detected, reported as NaN queries: an invalid tree, a slot outside
 * [0, slots) or of an earlier sequence of the call, a length outside the
 * page table, more rows than recent_rows - len % page_tokens (nothing of such
 * a sequence is written to the cache); a position outside [0, positions)
 * (that row's query, and its key's rotated dims).
 */
w12_status w12_kv_append(const w12_kv_cache *cache, int32_t layer, int32_t num_seq, const int32_t *slot,
                         const int32_t *row_off, int32_t total_rows, const int32_t *parent, const void *qkv,
                         int qkv_type, int32_t q_heads, const float *rope, int32_t positions, int32_t rot_dim,
                         int32_t interleaved, uint16_t *q, hipStream_t stream);

/* Workspace bytes w12_kv_attention needs (host output). */
w12_status w12_kv_attention_workspace(const w12_kv_cache *cache, int32_t num_seq, int32_t total_rows, int32_t q_heads,
                                      size_t *bytes);

/*
 * w12_kv_attention -- attention of a step's rows: row i attends to its
 * sequence's committed tokens and to its own ancestors among the step's rows,
 * itself included,
 *   out[i, h] = softmax(scale q[i, h] . K) V,  kv head h / (q_heads / kv_heads),
 *   scale > 0, finite,
 * with fp32 scores, sums and accumulation; probabilities and 8-bit codes
 * enter the matrix products as bf16 (the codes exactly, a probability off by
 * up to 2^-8 of itself, in the sum as in the product). Infinities and NaN
 * in rows that a row does not see never reach it. The split of long
 * sequences over workgroups is in a fixed order: results are bitwise
 * reproducible.
 *   q    [total_rows][q_heads][head_dim] bf16 (w12_kv_append's output).
 *   out  [total_rows][q_heads * head_dim] bf16: the x of the Wo product; not q's memory.
 *   ws   workspace of >= w12_kv_attention_workspace bytes, 256-byte aligned,
 *        content ignored; of one call at a time (two streams, two captured
 *        graphs, two host threads whose calls overlap: one each).
 * Device-detected, reported as NaN outputs of the sequence: what w12_kv_append
 * lists (a slot named twice is allowed here), and a page id outside
 * [0, num_pages). Weighted values are summed before they are normalised:
 * values beyond 2^100 may come out as infinities or NaN.
 */
w12_status w12_kv_attention(const w12_kv_cache *cache, int32_t layer, int32_t num_seq, const int32_t *slot,
                            const int32_t *row_off, int32_t total_rows, const int32_t *parent, const uint16_t *q,
                            int32_t q_heads, float scale, uint16_t *out, void *ws, size_t ws_bytes,
                            hipStream_t stream);

/*
 * w12_kv_commit -- keeps the accepted rows of a step, in all layers at once:
 * row path[0 .. accept_len] of each sequence (tree_accept's outputs: path
 * [total_rows], tree-local and ascending from the root; NULL: the first
 * accept_len + 1 rows) join its committed tokens in order. Every block that
 * becomes full is quantised into its page (page_table[slot][len / page_tokens
 * ...] must name pages for them): scale = the smallest power of two with
 * amax <= 448 scale (e4m3) or amax / 127 (int8), at least 2^-90, 1 for a block
 * of zeros; code = value / scale, rounded to nearest even. A block that holds
 * an infinity or NaN gets scale NaN. The rows left move to the front of the
 * recent rows.
 *   len_out [slots] out: the new length of each sequence's slot, other
 *           entries left as they are; may be the cache's own len.
 * accept_len -1 (a refused tree) keeps nothing. Device-detected, reported as
 * length -1 with nothing written (a slot named twice: its first sequence
 * stands): what w12_kv_append lists (trees aside), an
 * accept_len or path outside the sequence's rows or not ascending from row 0,
 * a page id outside [0, num_pages), a new length beyond max_pages *
 * page_tokens.
 */
w12_status w12_kv_commit(const w12_kv_cache *cache, int32_t num_seq, const int32_t *slot, const int32_t *row_off,
                         int32_t total_rows, const int32_t *accept_len, const int32_t *path, int32_t *len_out,
                         hipStream_t stream);

/*
 * Recurrent layers of the verify pass (gated delta rule; [S1] 4.2: most
 * layers of the target are recurrent, their state is recomputed along each
 * root path, without a snapshot for each node, and the accepted path is
 * replayed into it). Per layer a step calls w12_delta_append, then
 * w12_delta_rule; w12_delta_commit keeps the accepted rows of all layers.
 *   state [layers][slots][value_heads][key_dim][value_dim] fp32: the state S
 *         of each sequence's committed tokens (zeros: none);
 *   conv  [layers][slots][conv_width - 1][channels] bf16: the convolution's
 *         window, the last inputs of the committed tokens, oldest first
 *         (zeros: before the first token), channels = 2 key_heads key_dim +
 *         value_heads value_dim;
 * and what the rows of one step leave for the calls behind, by the step's row:
 *   raw   [layers][step_rows][channels] bf16: the convolution's inputs;
 *   kv    [layers][step_rows][key_heads key_dim + value_heads value_dim]
 *         bf16: key heads, value heads;
 *   gates [layers][step_rows][2][value_heads] fp32: g (log of the decay, <= 0)
 *         and beta (strength) of each value head;
 *   delta [layers][step_rows][value_heads][value_dim] fp32: what a row adds
 *         to the state, S += k delta^T.
 * Value head h goes with key head h / (value_heads / key_heads). The rows of
 * a step are described as for the KV cache above: row_off, slot, parent (NULL:
 * chains), at most 512 rows and at most step_rows. These four arrays belong
 * to one step at a time: two steps in flight have a description each, over
 * the same state and conv. A slot may be named by several sequences of a
 * step, except where a call keeps rows.
 * Sizes: key_dim and value_dim 64 or 128; value_heads a multiple of
 * key_heads, at most 256; conv_width 2, 3 or 4; layers <= 1024; slots <=
 * 2^20; step_rows <= 65536. All arrays 16-byte aligned, and apart.
 */
typedef struct w12_delta_cache {
  int32_t layers, slots, step_rows, key_heads, value_heads, key_dim, value_dim, conv_width;
  float *state;
  uint16_t *conv;
  uint16_t *raw;
  uint16_t *kv;
  float *gates;
  float *delta;
} w12_delta_cache;

/*
 * w12_delta_append -- the inputs of a recurrent layer's rows. With x_0 a
 * row's input (qkv, rounded to bf16), x_1 its parent's, and so on, past the
 * root the slot's window from its newest entry back,
 *   y[c] = conv_bias[c] + sum_t conv_weight[c][conv_width - 1 - t] x_t[c],
 *   s = y / (1 + e^-y); query and key heads: s / sqrt(sum s^2 + 1e-6);
 *   beta = 1 / (1 + e^-b),  g = -e^a_log log(1 + e^(a + dt_bias)),
 * in fp32; queries, keys and values rounded to bf16 once.
 *   qkv  [total_rows] rows of channels values, qkv_stride values apart (a
 *        multiple of 16 bytes): query heads, key heads, value heads;
 *   ba   [total_rows] rows of 2 value_heads values, ba_stride apart: b, then
 *        a; both fp32 or both bf16 (type a w12_ydtype): columns of one fused
 *        product as they lie;
 *   conv_weight [channels][conv_width] fp32, the row's own tap last;
 *   conv_bias [channels] fp32 or NULL; a_log, dt_bias [value_heads] fp32;
 *   q    [total_rows][key_heads][key_dim] bf16 out, apart from the cache's
 *        arrays and all that the call reads;
 * qkv, conv_weight, conv_bias and q 16-byte aligned.
 * Writes raw, kv and gates of its rows, which lie apart from all that the call
 * reads; state and conv are read at most.
 * Device-detected, reported as NaN queries with nothing staged: an invalid
 * tree, a slot outside [0, slots).
 */
w12_status w12_delta_append(const w12_delta_cache *cache, int32_t layer, int32_t num_seq, const int32_t *slot,
                            const int32_t *row_off, int32_t total_rows, const int32_t *parent, const void *qkv,
                            int64_t qkv_stride, const void *ba, int64_t ba_stride, int type, const float *conv_weight,
                            const float *conv_bias, const float *a_log, const float *dt_bias, uint16_t *q,
                            hipStream_t stream);

/*
 * w12_delta_rule -- the gated delta rule over the step's rows. Along a row's
 * root path, from its slot's state,
 *   S <- e^g S;  delta = beta (v - S^T k);  S <- S + k delta^T;
 *   out[i, h] = scale S^T q[i],  scale finite,
 * with fp32 states, deltas and accumulation (a factor that is not bf16 enters
 * the matrix products whole: in fp32, or in three bf16 pieces that hold its 24 bits)
 * and decays summed in 64 bits. A row sees its ancestors and itself: an
 * infinity or NaN in a row's k, v or gates (g of minus infinity apart: it
 * forgets the state) leaves no numbers in its own outputs and deltas, those of
 * the rows behind it on their paths, and the state behind them; in its q, none
 * in its own outputs. No other row's change. Of k, q and
 * the gates it reaches all of the value heads that they belong to; of v at least
 * the value dim it stands in and at most its head (how many of the head's other
 * dims share a workgroup goes by the form that the call takes). Deltas and
 * products beyond 2^100 may come out as infinities or NaN in the whole sequence.
 *   q    [total_rows][key_heads][key_dim] bf16 (w12_delta_append's output);
 *   out  [total_rows][value_heads * value_dim] bf16, apart from the cache's
 *        arrays and all that the call reads; q and out 16-byte aligned;
 *   keep 0: writes the rows' delta; state and conv stay, and w12_delta_commit
 *        keeps the accepted rows. Not 0 (parent NULL only: prompts, plain
 *        decoding): every row is kept, state and conv become those behind the
 *        last row, and delta is not written. q, slot, row_off and parent lie
 *        apart from what is written.
 * Device-detected, reported as NaN outputs of the sequence with nothing else
 * written: what w12_delta_append lists, and with keep a slot of an earlier
 * sequence of the call. Results are bitwise reproducible.
 * The kernel's form goes by the mean rows of a sequence, empty ones counted: a
 * step of single rows and long sequences is faster as two calls, each over its
 * own part of slot and row_off, the single rows first and the first call's
 * total_rows theirs alone.
 */
w12_status w12_delta_rule(const w12_delta_cache *cache, int32_t layer, int32_t num_seq, const int32_t *slot,
                          const int32_t *row_off, int32_t total_rows, const int32_t *parent, const uint16_t *q,
                          float scale, int32_t keep, uint16_t *out, hipStream_t stream);

/*
 * w12_delta_commit -- keeps the accepted rows of a step, in all layers at
 * once: rows path[0 .. accept_len] of each sequence (tree_accept's outputs, as
 * for w12_kv_commit; NULL: the first accept_len + 1 rows) join the state,
 *   S <- e^G_n S + sum_j e^(G_n - G_j) k_j delta_j^T,  G_j = g_0 + ... + g_j
 * along the path, and the window.
 *   kept [num_seq] out: rows kept; accept_len -1 (a refused tree) keeps none.
 *        Apart from the cache's arrays and all that the call reads, as state
 *        and conv are from the latter.
 * Device-detected, reported as kept -1 with nothing written: a slot outside
 * [0, slots) or of an earlier sequence, a range of rows that is none, an
 * accept_len or path outside the sequence's rows or not ascending from row 0.
 */
w12_status w12_delta_commit(const w12_delta_cache *cache, int32_t num_seq, const int32_t *slot, const int32_t *row_off,
                            int32_t total_rows, const int32_t *accept_len, const int32_t *path, int32_t *kept,
                            hipStream_t stream);

/*
 * w12_norm -- what stands between two products: the norm behind a block, its
 * gate, the residual and its scale, the norm before the next block. For each
 * row and each of its groups of width values, with rms(x) = x / sqrt(mean x^2
 * + eps) and every absent part left out,
 *   t = y;  t = rms(t) post_weight;  t = t gate / (1 + e^-gate);
 *   h = h + scale t, rounded to h's type;  out = rms(u) weight,
 * u = h as it is stored, or t where there is no h; out rounded to bf16 once,
 * all else in fp32. So the norm before a block is (y, h, weight); the gated
 * norm of a recurrent layer's heads (y, post_weight, gate) with groups =
 * value_heads; the product between Wgate|Wup and Wdown (y, gate).
 *   y    [rows] rows of groups * width values, y_stride values apart; NULL
 *        (with h): h stays as it is, and there is no post_weight and no gate;
 *   gate as y, or NULL; y_type and gate_type w12_ydtypes;
 *   h    [rows][groups * width], h_type a w12_ydtype, or NULL;
 *   post_weight, weight [width] fp32 or NULL; eps > 0, scale finite;
 *   out  [rows][groups * width] bf16. out, h and the inputs are apart.
 * rows <= 2^24, groups <= 1024, width <= 32768. Any width and stride; the
 * fastest where rows and groups begin at multiples of 16 bytes.
 */
w12_status w12_norm(int64_t rows, int32_t groups, int32_t width, const void *y, int y_type, int64_t y_stride,
                    const float *post_weight, const void *gate, int gate_type, int64_t gate_stride, float scale,
                    void *h, int h_type, const float *weight, float eps, uint16_t *out, hipStream_t stream);

/* Workspace bytes tree_accept_sampled needs (host output). */
w12_status tree_accept_sampled_workspace(int32_t num_trees, int32_t total_nodes, int32_t vocab, size_t *bytes);

/*
 * tree_accept_sampled -- tree verification of sampling requests: drafted
 * tokens against the target's probabilities, from given random numbers ([S3]
 * speculative sampling: accept with min(1, p / q), else draw from max(0, p -
 * q)). Trees as in tree_accept (at most 1024 nodes each, total_nodes and
 * num_trees at most 65535); row i of logits belongs to node i,
 *   p = softmax(logits[i] / temperature[tree]).
 * From the root, a node's children are tried in index order against what
 * the rejections so far have left of p: child c with token x is accepted, and
 * the walk goes on from it, if u_accept[c] q(x) < p(x); otherwise p becomes
 * max(p - q, 0), normalised. q = draft[i] (the distribution that node i's
 * children were drawn from), or, with draft NULL, one at x (drafts that were
 * chosen, not drawn). Where no child is accepted the walk ends, and the bonus
 * token is the lowest t whose cumulative sum of p exceeds u_bonus[tree] times
 * the whole sum (the last token with p > 0 if none does). The tokens that come
 * out are distributed as if drawn from the target alone.
 * Probabilities, sums and comparisons are held in 64 bits; an exponential
 * e^-a is off by up to 2e-15 + 2e-16 a of itself, some of its last bits.
 *   logits  [total_nodes][vocab] fp32 or bf16 (logits_type a w12_ydtype),
 *           w12_gemm's y of the head; vocab <= 2^28.
 *   temperature [num_trees] fp32 > 0, or NULL (1); draft [total_nodes][vocab]
 *           fp32 or NULL (rows of nodes without children are not read);
 *   u_accept [total_nodes], u_bonus [num_trees] fp32 in [0, 1).
 *   accept_len, path, bonus: as tree_accept's.
 *   ws      workspace, 16-byte aligned, content ignored; of one call at a time.
 * Device-detected, reported as accept_len = bonus = -1 and a path of -1: what
 * tree_accept lists, a drafted token outside [0, vocab), more than 1024
 * nodes, a temperature that is not positive and finite, and a row on the walk
 * whose logits hold NaN, +inf or nothing but -inf.
 */
w12_status tree_accept_sampled(int32_t num_trees, const int32_t *node_off, int32_t total_nodes, const int32_t *parent,
                               const int32_t *token, const void *logits, int logits_type, int32_t vocab,
                               const float *temperature, const float *draft, const float *u_accept,
                               const float *u_bonus, int32_t *accept_len, int32_t *path, int32_t *bonus, void *ws,
                               size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* W12_H */
