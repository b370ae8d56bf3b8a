/*
 * jsv.h -- C ABI of libjsv.so: the one-forward tree verification step of
 * causal parallel tree drafting (JetSpec), as hand-written CUDA for sm_100a.
 *
 * The method (JetSpec README, "JetSpec / Overview"): a draft head proposes a
 * token tree; the frozen target verifies the whole tree in ONE forward pass
 * under a tree-causal attention mask, and the accepted path is chosen by the
 * target's own logits, so decoding stays lossless.  The serving engine keeps
 * the KV cache in pages (README, "JetSpec / Quick Start": paged KV, custom
 * tree attention, CUDA graphs).  All reported runs are greedy (temperature 0).
 * One verify step is four calls on one stream, in this order:
 *
 *   jsv_tree_attention  tree-causal attention of every node over its
 *                       request's paged KV prefix plus its own ancestors
 *   jsv_lmhead_argmax   LM-head projection of every node's hidden state
 *                       fused with top-1 argmax (logits are never stored)
 *   jsv_accept_path     greedy longest-accepted-path walk
 *   jsv_kv_compact      move the accepted path's K/V rows to contiguous
 *                       slots P..P+a of each request (ragged batches)
 *
 * jsv_accept_compact does the last two in one launch.  Over a prefix held in
 * 8 bits jsv_tree_attention_kv8 takes the first call's place; the page pool's
 * calls (jsv_pages_*) and jsv_kv8_quantize turn the pages over between steps.
 *
 * Conventions for every call
 *   - Pointers marked "device" are CUDA device (or managed) memory; the
 *     caller allocates and owns every buffer, workspace included.  The
 *     library never allocates, frees or synchronises.
 *   - bf16 tensors are IEEE bfloat16 bit patterns, row-major, contiguous.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Calls
 *     are asynchronous: the return value covers host-side argument checks
 *     and the launch only.
 *   - Host-side checks return JSV_ERR_INVALID_ARG (NULL pointer, negative or
 *     inconsistent size, too-small workspace) or JSV_ERR_UNSUPPORTED (a
 *     shape outside the supported set) and launch nothing.
 *   - Errors that only the device can see (a malformed parent array, a page
 *     index outside [0, num_pages), node offsets that disagree with
 *     total_nodes, a path longer than max_path) are written to
 *     batch->dev_status (if non-NULL) with an atomic compare-and-swap from
 *     0, so the first error sticks; the affected request's work is skipped.
 *     Kernels never trap.  The caller zeroes *dev_status before a step.
 *   - Calls on distinct streams with distinct workspaces and outputs may run
 *     concurrently.
 */
#ifndef JSV_H
#define JSV_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define JSV_API __attribute__((visibility("default")))
#else
#define JSV_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    JSV_OK = 0,
    JSV_ERR_INVALID_ARG = 1,   /* host-visible bad argument                  */
    JSV_ERR_UNSUPPORTED = 2,   /* shape outside the supported set            */
    JSV_ERR_CUDA = 3,          /* a CUDA runtime call or launch failed       */
    JSV_ERR_TIMEOUT = 4,       /* a bounded device wait gave up              */
    JSV_ERR_DEVICE_INPUT = 5,  /* written to *dev_status: bad device data    */
    JSV_ERR_BOUNDS = 6,        /* written to *dev_status, only by a library
                                  built with JSV_CHECK_BOUNDS: a computed
                                  index fell outside its buffer (a library
                                  fault; the access was skipped)            */
    JSV_ERR_NO_PAGES = 7       /* written to *dev_status: a page pool had too
                                  few free pages for a request, which was
                                  left as it was                            */
} jsv_status;

/*
 * Geometry of one verify step over B requests, shared by the calls that
 * touch the tree or the cache.
 *
 * Notation: request b has P_b committed prefix tokens and a draft tree of
 * N_b nodes (node 0 = root = the last committed token, whose K/V this
 * forward computes).  Nodes of all requests are packed: request b owns
 * global nodes node_offsets[b] .. node_offsets[b+1]-1, T = node_offsets[B].
 *
 * Tree: parent[] holds request-local indices with parent[0] = -1 and
 * 0 <= parent[i] < i for i > 0 (any topological order).
 *
 * Cache: k_cache and v_cache are [num_pages][page_size][Hkv][D] bf16.
 * Logical slot s of request b is row s % page_size of physical page
 * page_table[b * max_pages_per_req + s / page_size].  Slots [0, P_b) hold
 * the prefix; the caller has written tree node j's K/V at slot P_b + j, so
 * pages covering [0, P_b + N_b) must be mapped.
 */
typedef struct {
    int32_t B;                   /* requests, >= 1                                */
    int32_t Hq, Hkv, D;          /* query heads, KV heads (Hq % Hkv == 0), D in {64,128} */
    int32_t page_size;           /* must be 16                                    */
    int32_t max_pages_per_req;   /* row stride of page_table                      */
    int32_t num_pages;           /* physical pages in k_cache and in v_cache      */
    int32_t total_nodes;         /* T, must equal node_offsets[B]                 */
    int32_t max_nodes;           /* upper bound on N_b, 1..512                    */
    int32_t max_prefix;          /* upper bound on P_b, >= 0                      */
    const int32_t *page_table;   /* device [B][max_pages_per_req]                 */
    const int32_t *prefix_len;   /* device [B]   P_b                              */
    const int32_t *node_offsets; /* device [B+1]                                  */
    const int32_t *parent;       /* device [T]   request-local parent index       */
    int32_t *dev_status;         /* device [1] or NULL: first device-side error   */
} jsv_batch;

/* Bytes of scratch jsv_tree_attention needs for this geometry (split-KV
 * partial results; 0 when every request takes one split).  Depends on the
 * host-side fields and on the current device's SM count, which sets the
 * split count. */
JSV_API size_t jsv_tree_attention_workspace_size(const jsv_batch *batch);

/*
 * Tree-causal attention (README, "JetSpec / Overview": one forward pass under
 * a tree-causal mask).  For request b, node i, query head h, with
 * g = h / (Hq / Hkv), the visible sequence is prefix slots 0..P_b-1 followed
 * by slots P_b + j for every j on the root..i path (i included):
 *     out[t][h] = sum_j softmax_j(scale * <q[t][h], k_j>) * v_j
 * computed in fp32 from bf16 inputs and rounded to bf16.
 *   q        device [T][Hq][D] bf16, post-rotary
 *   k_cache, v_cache  device caches as described above (read only)
 *   scale    softmax scale (normally 1/sqrt(D))
 *   out      device [T][Hq][D] bf16
 *   workspace, workspace_bytes  device scratch of at least
 *            jsv_tree_attention_workspace_size(batch) bytes, 256-B aligned
 *            (NULL is accepted when that size is 0); any contents, since
 *            every call writes what it reads
 */
JSV_API jsv_status jsv_tree_attention(const jsv_batch *batch, const uint16_t *q,
                              const uint16_t *k_cache, const uint16_t *v_cache,
                              float scale, uint16_t *out,
                              void *workspace, size_t workspace_bytes, void *stream);

/*
 * Budgeted draft-tree construction by cumulative log-probability (the pages'
 * default "accum_logp" tree: JetSpec README, "Evaluation", breadth-first and
 * kept by cumulative log-probability under depth, width and budget).  Reading:
 * for each request the draft head gives, per depth m = 1..depth, its top-width
 * candidate tokens with log-probabilities sorted in descending order.  A node
 * is a rank path; its score is the fp32 running sum of its edge log-probs
 * (added root to leaf).  The tree is the `budget` best nodes under
 *     score descending, depth ascending, rank path lexicographic ascending
 * (root = empty path, score 0, always kept), in breadth-first order with
 * children in rank order: parent[0] = -1 and parent[i] < i, ready for the
 * other calls.
 *   logp         device [B][depth][width] float, each row non-increasing, <= 0
 *   topk_tokens  device [B][depth][width] int32
 *   root_token   device [B] int32 (the last committed token)
 *   parent, tokens, node_depth  device [B][budget] int32 outputs; slots past
 *                num_nodes[b] get -1
 *   score        device [B][budget] float or NULL (fp32 node scores)
 *   num_nodes    device [B] int32: nodes emitted (budget, or fewer when the
 *                whole candidate tree is smaller)
 *   dev_status   device [1] int32 or NULL: a request whose log-probs are not
 *                sorted, positive or NaN gets JSV_ERR_DEVICE_INPUT and a
 *                root-only tree
 * Supported: 1 <= B, 0 <= depth <= 32, 1 <= width <= 32, 1 <= budget <= 512.
 */
JSV_API jsv_status jsv_accum_logp_tree(const float *logp, const int32_t *topk_tokens,
                                       const int32_t *root_token, int32_t B, int32_t depth,
                                       int32_t width, int32_t budget, int32_t *parent,
                                       int32_t *tokens, int32_t *node_depth, float *score,
                                       int32_t *num_nodes, int32_t *dev_status, void *stream);

/*
 * Tree Q/K/V projection with rotary positions, K/V appended to the paged cache
 * (the step before jsv_tree_attention; reading of the JetSpec README,
 * "JetSpec / Overview" and "Quick Start": one forward pass over the tree,
 * paged KV).  For node j of request b, qkv = w_qkv x_j with rows Q heads
 * (Hq*D), then K heads (Hkv*D), then V heads (Hkv*D); Q and K heads are
 * rotated at position P_b + depth(j) with the rotate-half pairs (i, i + D/2):
 *     out_i = x_i c_i - x_{i+D/2} s_i,  out_{i+D/2} = x_{i+D/2} c_i + x_i s_i
 * Q is written to q[j], K and V to logical slot P_b + j of the request's
 * pages.  fp32 accumulation, bf16 outputs.
 *   x          device [T][d] bf16 (the tree's hidden states entering the layer)
 *   w_qkv      device [(Hq + 2 Hkv) D][d] bf16
 *   rope_cos, rope_sin  device [max_pos][D/2] float tables
 *   q          device [T][Hq][D] bf16 output
 *   k_cache, v_cache  the paged caches; only tree slots P_b .. P_b+N_b-1 change
 * A node whose position reaches max_pos, or whose parent chain or page is
 * malformed, is skipped and JSV_ERR_DEVICE_INPUT is written to dev_status.
 * Supported: d % 64 == 0, 64 <= d <= 16384.
 */
JSV_API jsv_status jsv_tree_qkv_rope(const jsv_batch *batch, const uint16_t *x, const uint16_t *w_qkv,
                                     int32_t d, const float *rope_cos, const float *rope_sin,
                                     int32_t max_pos, uint16_t *q, uint16_t *k_cache,
                                     uint16_t *v_cache, void *stream);

/* Bytes of scratch jsv_lmhead_argmax needs (one 64-bit key per node and a
 * completion counter). */
JSV_API size_t jsv_lmhead_argmax_workspace_size(int32_t T, int32_t d, int32_t V);

/*
 * LM head fused with top-1 argmax (README, "JetSpec / Overview": the path is
 * selected by the target's own logits; temperature 0).
 *     argmax[t] = smallest v attaining max_v sum_k hidden[t][k] * w[v][k]
 * accumulated in fp32 from bf16; logits are never written to memory.
 *   hidden     device [T][d] bf16
 *   w          device [V][d] bf16 (the LM-head weight, row per token)
 *   argmax     device [T] int32
 *   max_logit  device [T] float (the fp32 maximum) or NULL
 *   workspace  device scratch of jsv_lmhead_argmax_workspace_size() bytes,
 *              8-B aligned, ZERO-FILLED before its first use (e.g. one
 *              cudaMemsetAsync when it is allocated); every call leaves it
 *              zero-filled again, so it is reused without clearing.
 *   dev_status device [1] int32 or NULL.  A bounded wait of the kernel that
 *              gave up writes JSV_ERR_TIMEOUT (compare-and-swap from 0); the
 *              call's argmax and max_logit are then unspecified, and the
 *              workspace is still left zero-filled (every CTA counts the work
 *              it took, finished or abandoned, and the CTA that completes the
 *              count clears the keys and the counter).
 * Ordering: the kernel reads `hidden` and `w` while the previous launch on
 * the stream may still be running (it waits for that launch only before it
 * touches the workspace and the outputs), so the tree-attention kernels of
 * the same step run beside its main loop.  Kernels of other libraries are
 * complete before it starts, as usual; only a buffer written by an earlier
 * call of THIS library that may still be in flight (for instance
 * jsv_tree_attention's `out`) must not be passed as `hidden` or `w`.
 * Supported: 1 <= T, d % 64 == 0, 64 <= d <= 16384, 1 <= V < 2^31.
 */
JSV_API jsv_status jsv_lmhead_argmax(const uint16_t *hidden, const uint16_t *w,
                             int32_t T, int32_t d, int32_t V,
                             int32_t *argmax, float *max_logit,
                             void *workspace, size_t workspace_bytes,
                             int32_t *dev_status, void *stream);

/*
 * Greedy accept walk (README, "JetSpec / Overview": lossless by
 * construction; "tokens per forward" = accepted + 1).  Per request, start at
 * the root (always accepted); while some child c of the current node has
 * tokens[c] == argmax[current], move to the smallest such c.
 *   tokens      device [T] int32, the draft token of every node
 *   argmax      device [T] int32, the target's choice at every node
 *   max_path    row length of `path` (>= 1)
 *   path        device [B][max_path] int32: request-local indices of the
 *               accepted path starting with 0, then -1 padding
 *   accept_len  device [B] int32: accepted draft nodes a = path length - 1
 *   bonus       device [B] int32: argmax at the last accepted node
 * A path that would exceed max_path sets JSV_ERR_DEVICE_INPUT and is cut.
 */
JSV_API jsv_status jsv_accept_path(const jsv_batch *batch, const int32_t *tokens,
                           const int32_t *argmax, int32_t max_path,
                           int32_t *path, int32_t *accept_len, int32_t *bonus,
                           void *stream);

/*
 * Accepted-path KV compaction (README, "JetSpec / Quick Start": paged KV).
 * For every request and k = 0..a: the K and V rows (all KV heads) of slot
 * P_b + path[k] move to slot P_b + k, with the result of an in-order copy
 * (every source is read before any destination is written).  Slots other
 * than P_b..P_b+a are untouched.  new_len[b] = P_b + a + 1.
 *   k_cache, v_cache  device caches, updated in place
 *   path, accept_len  as written by jsv_accept_path (max_path = row stride)
 *   new_len           device [B] int32
 */
JSV_API jsv_status jsv_kv_compact(const jsv_batch *batch, uint16_t *k_cache, uint16_t *v_cache,
                          const int32_t *path, int32_t max_path, const int32_t *accept_len,
                          int32_t *new_len, void *stream);

/*
 * jsv_accept_path followed by jsv_kv_compact, in one kernel launch: the
 * step's two latency-bound tail calls fused (the pages have no counterpart;
 * a deployment form of the same two operations).  Every output -- path,
 * accept_len, bonus, the K/V caches and new_len -- and every device-side
 * error equals what the two calls in sequence produce on the same inputs.
 * Arguments follow those two calls: the tree arrays and argmax are read, the
 * path row is written with stride max_path, and the caches are updated in
 * place.  Every argument, the batch geometry included, is read only after
 * the previous launch on the stream has completed, so new_len of one step
 * may be passed back as the next step's prefix_len.
 */
JSV_API jsv_status jsv_accept_compact(const jsv_batch *batch, const int32_t *tokens,
                                      const int32_t *argmax, int32_t max_path,
                                      int32_t *path, int32_t *accept_len, int32_t *bonus,
                                      uint16_t *k_cache, uint16_t *v_cache, int32_t *new_len,
                                      void *stream);

/*
 * LM head fused with top-1 argmax for callers that cannot allocate device
 * memory (a region under CUDA-graph capture, a plugin whose host owns every
 * allocation, a loop that cannot afford cudaMalloc's synchronisation).
 * The pages have no counterpart: it is a deployment variant of
 * jsv_lmhead_argmax with the same result, whose scratch (one 64-bit key per
 * node) is a fixed file-scope device array inside the library instead of a
 * workspace argument.  The caller still passes inputs and outputs.
 *   - T must be <= JSV_NOALLOC_MAX_NODES, else JSV_ERR_UNSUPPORTED; the
 *     other arguments, dev_status included, follow jsv_lmhead_argmax.
 *   - The array ((JSV_NOALLOC_MAX_NODES + 1) * 8 bytes) is held on every GPU
 *     that loads the library until the process exits.
 *   - The first call on a device looks up the array's device address (with
 *     that device current) and caches it; make that first call before any
 *     stream capture.
 *   - Nothing is allocated or freed: no cudaMalloc, cudaFree or allocating
 *     library routine.  The array starts zeroed and every call leaves the
 *     keys it used and the counter zeroed again, a call that reported
 *     JSV_ERR_TIMEOUT included (its outputs are then unspecified).
 *   - Every call shares the one array, which keeps the last call's contents:
 *     calls whose kernels overlap on the GPU (different streams, or
 *     different host threads on one device) race and give wrong results.
 *     Serialise them on one stream.
 */
#define JSV_NOALLOC_MAX_NODES 8192
JSV_API jsv_status jsv_lmhead_argmax_noalloc(const uint16_t *hidden, const uint16_t *w,
                                             int32_t T, int32_t d, int32_t V,
                                             int32_t *argmax, float *max_logit,
                                             int32_t *dev_status, void *stream);

/*
 * 8-bit key/value cache.  The full 16-slot pages of a request's committed
 * prefix are held as 8-bit codes with one fp32 scale for each (page, KV head)
 * of K and of V; the last, partial page and the tree's slots stay in the bf16
 * cache.  For request b with P_b prefix tokens:
 *     slots [0, 16 * floor(P_b / 16))          8-bit pages, jsv_kv8.page_table
 *     slots [16 * floor(P_b / 16), P_b + N_b)  bf16 pages, jsv_batch.page_table
 * Both tables are indexed by logical page (slot / 16); jsv_batch.page_table
 * entries below floor(P_b / 16) are not read, so their bf16 pages may be
 * freed or shared out again.  A value is code * scale; scales are not
 * negative, and V scales below 1e-37, or below 2^-64 of another of the same
 * request and head, may count as zero.
 * Layout: codes [num_pages][Hkv][16][D] (the 16 x D block of one page and
 * head is contiguous), scales [num_pages][Hkv]; num_pages * Hkv * 16 < 2^31.
 * The pages that the README's engine keeps are bf16; this is a deployment
 * form of the same cache with half its bytes.  Attention over it is also
 * faster than over bf16 where few rows read much (one token a request 2.2 to
 * 3.6 times, 8 nodes 1.1 to 1.2 times), and slower where many rows do: 64
 * nodes over 2,048 tokens and more take 1.2 to 1.5 times as long, since the
 * codes are converted beside the products.  Device pointers of these and
 * the page pool's calls belong to the current device, whose stream is given.
 */
typedef enum {
    JSV_KV8_E4M3 = 0,            /* 4-bit exponent, 3-bit mantissa, largest 448 */
    JSV_KV8_INT8 = 1             /* two's complement, -128..127                 */
} jsv_kv8_format;

typedef struct {
    int32_t format;              /* jsv_kv8_format                                */
    int32_t num_pages;           /* physical pages in k and in v                  */
    int32_t max_pages_per_req;   /* row stride of page_table                      */
    uint8_t *k, *v;              /* device [num_pages][Hkv][16][D] codes, 16-B aligned */
    float *k_scale, *v_scale;    /* device [num_pages][Hkv]                       */
    const int32_t *page_table;   /* device [B][max_pages_per_req]                 */
} jsv_kv8;

/* Bytes of scratch jsv_tree_attention_kv8 needs for this geometry (split-KV
 * partial results).  Depends on the host-side fields of both structures and
 * on the current device's SM count; 0 when no request is split. */
JSV_API size_t jsv_tree_attention_kv8_workspace_size(const jsv_batch *batch, const jsv_kv8 *cache8);

/*
 * Tree-causal attention as jsv_tree_attention defines it, over a prefix whose
 * full pages are read from the 8-bit cache (the last, partial page and the
 * tree's own slots from the bf16 caches).  One node per request (node 0
 * alone) is ordinary single-token decoding.  Scores, softmax statistics and
 * the output are accumulated in fp32; the output is rounded to bf16.  In the
 * products the weight of a key of an 8-bit page is held to 2^-11 of itself or
 * 2^-25 of the row's largest weight, whichever is more, and a V value to 2^-10
 * of itself and 2^-29 of the largest V scale among the eight pages of its 128
 * slots; weights of bf16 pages are rounded to bf16.
 * How a request is split is chosen on the host, by max_prefix, max_nodes and
 * the two caches' pages: results depend on how near these bounds are by fp32
 * rounding only, times by up to twice.
 *   q, scale, out, stream   as for jsv_tree_attention (scale <= 2.3e38)
 *   k_cache, v_cache        the bf16 caches (batch->num_pages pages)
 *   workspace, workspace_bytes  device scratch of at least
 *            jsv_tree_attention_kv8_workspace_size() bytes, 256-B aligned
 *            (NULL is accepted when that size is 0); any contents, written
 *            and read within the call: calls that may overlap, graphs
 *            replayed side by side included, take workspaces of their own
 * Values that a node does not see do not reach its output, whatever they are
 * (infinities and NaN in later slots of a page and in other branches of the
 * tree included).  A node that sees a non-finite V value or scale, however
 * small its weight, gets non-finite outputs (a visible non-finite value in the
 * bf16 V cache makes all of the head's output NaN); so does one that sees a
 * NaN in K or a non-finite K scale.  An infinity in the bf16 K cache counts by
 * its score: plus infinity gives NaN, minus infinity a weight of zero, and NaN
 * where no score of the node is finite.
 * Supported: D in {64, 128}, B * Hkv <= 65535; prefix pages need a row in
 * each table.  The codes of a request's pages are trusted; page indices are
 * checked.
 */
JSV_API jsv_status jsv_tree_attention_kv8(const jsv_batch *batch, const jsv_kv8 *cache8, const uint16_t *q,
                                          const uint16_t *k_cache, const uint16_t *v_cache, float scale,
                                          uint16_t *out, void *workspace, size_t workspace_bytes, void *stream);

/*
 * How jsv_tree_attention_kv8 takes a geometry on the current device, from the
 * host-side fields of both structures: a diagnostic for tests and for the
 * choice of bounds (a batch whose prefixes stay far below max_prefix, or a
 * pool with many pages to spare, gets fewer splits than it could use).
 */
typedef struct {
    int32_t rows;                /* query rows of a KV head that are taken together:
                                    8 or 16 (streaming form) or 256 (tcgen05 form)     */
    int32_t splits;              /* most splits of a request                           */
    int32_t split_units;         /* pages (streaming) or 128-slot tiles that a split
                                    aims at                                            */
} jsv_kv8_plan;
JSV_API jsv_status jsv_tree_attention_kv8_plan(const jsv_batch *batch, const jsv_kv8 *cache8, jsv_kv8_plan *plan);

/*
 * Full pages of the bf16 cache written to the 8-bit cache.  For request b the
 * logical pages floor(from_len[b] / 16) .. floor(to_len[b] / 16) - 1 are read
 * through batch->page_table and written through cache8->page_table: after a
 * prefill from_len is NULL (zeros) and to_len the prompt lengths; after a
 * verify step from_len is the old prefix_len and to_len the compaction's
 * new_len.  Per (page, KV head), of K and of V:
 *     scale = amax / qmax,  code = round(x * qmax / amax)
 * with amax = max |x| over the block's 16 x D values, qmax = 448 (e4m3) or
 * 127 (int8), the quotient taken in fp32 and rounded to nearest, ties to
 * even; a block of zeros has scale 0 and zero codes.  A block with an
 * infinity or NaN is written with scale NaN and zero codes, and
 * JSV_ERR_DEVICE_INPUT goes to dev_status.  Other pages of the 8-bit cache
 * are left as they are.  Of the batch, B, Hkv, D, num_pages, the page table
 * and dev_status are used (the other fields are checked on the host as for any
 * call).  A request whose lengths are not
 * 0 <= from_len <= to_len or need a page past either table's row, or a page
 * whose entry is out of range, is flagged (JSV_ERR_DEVICE_INPUT) and skipped.
 * Two requests must not write the same 8-bit page in one call; one that asks
 * for more pages than the cache has is flagged and writes nothing.
 * Supported: B <= JSV_PAGES_MAX_ROWS, B * cache8->max_pages_per_req < 2^31.
 *   from_len, to_len   device [B] int32 (from_len may be NULL)
 */
#define JSV_PAGES_MAX_ROWS 8192
JSV_API jsv_status jsv_kv8_quantize(const jsv_batch *batch, const jsv_kv8 *cache8, const uint16_t *k_cache,
                                    const uint16_t *v_cache, const int32_t *from_len, const int32_t *to_len,
                                    void *stream);

/*
 * Page pool.  The library's calls take page tables as given; these calls
 * fill and empty them on the device, with no host round trip and in graph
 * capture.  A pool is num_pages physical pages (of every buffer that shares
 * the table: the K and V caches of all layers) and one reference count for
 * each: 0 = free, n = n page-table entries hold it.  The caller zero-fills
 * refcount once.  A table is [B][max_pages_per_req] int32, -1 = unmapped.
 * A free page is always taken lowest index first and requests are served in
 * row order, so the result depends on nothing but the inputs.  Full pages
 * are never written again, so rows may share them; a partial page is held by
 * one row.  Calls on one pool are issued on one stream.
 * Supported: B <= JSV_PAGES_MAX_ROWS; lengths are in slots, at most
 * 16 * max_pages_per_req (a row outside that is flagged with
 * JSV_ERR_DEVICE_INPUT and skipped).
 */
typedef struct {
    int32_t num_pages;
    int32_t *refcount;           /* device [num_pages]                            */
    int32_t *dev_status;         /* device [1] or NULL: first device-side error   */
} jsv_page_pool;

/* Bytes of scratch for jsv_pages_alloc, jsv_pages_fork and
 * jsv_pages_compact on a pool of num_pages pages and tables of B rows or
 * forks; 16-B aligned, any contents, written and read within the call. */
JSV_API size_t jsv_pages_workspace_size(int32_t num_pages, int32_t B);

/*
 * Map fresh pages: every unmapped entry of row b among the logical pages
 * floor(begin[b] / 16) .. ceil(end[b] / 16) - 1 gets a free page (reference
 * count 1); with full_only != 0 the range ends at floor(end[b] / 16) (the
 * pages that end[b] slots fill).  Rows are served in order while the pages
 * last: a row whose pages do not fit after all that the rows before it ask
 * for is left as it was and JSV_ERR_NO_PAGES is written to dev_status.
 *   page_table   device [B][max_pages_per_req], updated
 *   begin, end   device [B] int32 (begin may be NULL: zeros)
 */
JSV_API jsv_status jsv_pages_alloc(const jsv_page_pool *pool, int32_t *page_table, int32_t B,
                                   int32_t max_pages_per_req, const int32_t *begin, const int32_t *end,
                                   int32_t full_only, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Fork rows: for i = 0..n-1, row dst[i] becomes a copy of the first len[i]
 * slots of row src[i].  The floor(len / 16) full pages are shared (unmapped
 * entries stay unmapped); a partial page gets a fresh page for dst and the
 * pair goes to copy_src[i], copy_dst[i] for jsv_pages_copy (-1, -1 where
 * nothing is to be copied).  With full_only != 0 the partial page is left
 * out (a table of 8-bit pages, which are always full).
 * Row dst must be wholly unmapped and appear once among dst, and row src be
 * no fork's dst; else, and where the partial page of src is unmapped or an
 * entry is out of range or free, fork i is skipped and JSV_ERR_DEVICE_INPUT
 * written (of forks with the same dst the first is made; a fork into a row
 * that another names as its src is made, the other is not).  A fork that does
 * not get its page is skipped with JSV_ERR_NO_PAGES.
 *   src, dst, len        device [n] int32, 0 <= n <= JSV_PAGES_MAX_ROWS
 *   copy_src, copy_dst   device [n] int32
 */
JSV_API jsv_status jsv_pages_fork(const jsv_page_pool *pool, int32_t *page_table, int32_t B,
                                  int32_t max_pages_per_req, int32_t n, const int32_t *src, const int32_t *dst,
                                  const int32_t *len, int32_t full_only, int32_t *copy_src, int32_t *copy_dst,
                                  void *workspace, size_t workspace_bytes, void *stream);

/*
 * Free pages: of row b the logical pages floor(keep_begin[b] / 16) ..
 * ceil(keep_end[b] / 16) - 1 stay; every other mapped entry is unmapped and
 * its page's reference count falls by one (free at 0).  keep_begin NULL =
 * zeros: what lies past keep_end goes.  keep_begin = keep_end = new_len
 * leaves the partial page alone: what a bf16 table keeps once its full pages
 * are in the 8-bit cache.  keep_end = 0 empties the row.  An entry whose page
 * is out of range or already free is unmapped and flagged.
 */
JSV_API jsv_status jsv_pages_trim(const jsv_page_pool *pool, int32_t *page_table, int32_t B,
                                  int32_t max_pages_per_req, const int32_t *keep_begin, const int32_t *keep_end,
                                  void *stream);

/*
 * Plan a compaction: with U pages in use, every used page at index >= U moves
 * to a free page below U, both in ascending order, so that the used pages
 * become 0 .. U-1 (the pool's end can be handed back).  Nothing of the input
 * changes (page_table may equal new_table): after jsv_pages_copy has moved
 * the contents, the caller goes on with the new table and counts.
 *   new_table            device [B][max_pages_per_req] output
 *   new_refcount         device [num_pages] output
 *   copy_src, copy_dst   device [max_copies] output, -1 past the last pair
 *   max_copies           at least num_pages / 2 (the most pages that can move)
 *   num_copies           device [1] output
 * A table entry whose page is out of range or free becomes -1 and is flagged.
 */
JSV_API jsv_status jsv_pages_compact(const jsv_page_pool *pool, const int32_t *page_table, int32_t B,
                                     int32_t max_pages_per_req, int32_t *new_table, int32_t *new_refcount,
                                     int32_t *copy_src, int32_t *copy_dst, int32_t max_copies, int32_t *num_copies,
                                     void *workspace, size_t workspace_bytes, void *stream);

/*
 * Copy page contents in every buffer that shares the pool: for each pair
 * i < n (and < *num_copies where given) with copy_src[i] >= 0, page
 * copy_src[i] of every buffer is copied to page copy_dst[i].  No destination
 * may appear twice or be a source (the lists of jsv_pages_fork and
 * jsv_pages_compact are so).  A pair out of range is flagged and skipped.
 *   buffers      host array [n_buffers] of device addresses (page 0), read
 *                before the call returns; 4-B aligned, 16-B aligned copies
 *                faster
 *   page_bytes   host array [n_buffers]: bytes of one page, multiples of 4
 *   copy_src, copy_dst, num_copies   device (num_copies may be NULL)
 */
JSV_API jsv_status jsv_pages_copy(const jsv_page_pool *pool, void *const *buffers, const int64_t *page_bytes,
                                  int32_t n_buffers, const int32_t *copy_src, const int32_t *copy_dst, int32_t n,
                                  const int32_t *num_copies, void *stream);

/* Number of kernels this library has launched in the calling process since
 * it was loaded (all devices, all streams).  A diagnostic for counting the
 * launches inside a timed region; not tied to any stream order. */
JSV_API uint64_t jsv_kernel_launches(void);

/*
 * Failure-detection self-test of the bounded device waits.  Every wait of
 * the library's tensor-core kernels on an mbarrier gives up after a time
 * limit, writes JSV_ERR_TIMEOUT to the status word and unwinds (copies in
 * flight drained, TMEM released), so a lost arrival ends in a readable status
 * rather than a hung GPU.  This call launches one CTA that waits on a barrier
 * nothing signals, with the limit shortened to `limit_us` microseconds
 * (1 .. 2,000,000); it writes JSV_ERR_TIMEOUT to *dev_status (device int32,
 * compare-and-swap from 0) and exits, leaving the context usable.
 */
JSV_API jsv_status jsv_selftest_wait_timeout(int32_t *dev_status, uint32_t limit_us, void *stream);

/*
 * Failure-detection self-test of the LM head's timeout path.  Runs the LM head
 * exactly as jsv_lmhead_argmax does with `workspace` (or, with workspace
 * NULL, as jsv_lmhead_argmax_noalloc does, on the library's scratch array),
 * except that the producer warp of the first CTA -- the first CTA pair for
 * trees above 128 nodes -- first waits on a barrier that nothing signals,
 * with the limit shortened to `limit_us` microseconds (1 .. 2,000,000).  That
 * wait gives up before the CTA has issued any copy: the CTA writes
 * JSV_ERR_TIMEOUT to *dev_status (device int32, required, compare-and-swap
 * from 0), stops, and the rest of the grid completes.  argmax and max_logit
 * are then unspecified; the workspace (or scratch array) is left zeroed, so
 * the next ordinary call on it returns the right result.  Other arguments
 * and checks follow jsv_lmhead_argmax (and the T limit of the no-alloc form).
 */
JSV_API jsv_status jsv_selftest_lmhead_timeout(const uint16_t *hidden, const uint16_t *w,
                                               int32_t T, int32_t d, int32_t V,
                                               int32_t *argmax, float *max_logit,
                                               void *workspace, size_t workspace_bytes,
                                               int32_t *dev_status, uint32_t limit_us, void *stream);

/* Text of the last CUDA error behind a JSV_ERR_CUDA returned to the calling
 * host thread (a launch or runtime call that failed), or a fixed message if
 * none was recorded; for a failed kernel launch it also names the kernel's
 * registers and shared memory against the launch.  The string belongs to the
 * calling thread and stays valid until its next call; later successful calls
 * do not clear it. */
JSV_API const char *jsv_last_error_string(void);

/* Static string for a status code. */
JSV_API const char *jsv_status_string(jsv_status status);

/* Library version, major * 10000 + minor * 100 + patch. */
JSV_API int32_t jsv_version(void);

/* Build flags of this library: bit 0 set when it was compiled with
 * JSV_CHECK_BOUNDS (libjsv_checked.so), i.e. every computed global index
 * of the kernels is compared with its buffer's extent before the access and
 * a miss is skipped and written to the status word as JSV_ERR_BOUNDS.  The
 * pages have no counterpart: it is a debugging aid of this library. */
JSV_API int32_t jsv_build_flags(void);

#ifdef __cplusplus
}
#endif

#endif /* JSV_H */
