/*
 * kvsel — window-attention prompt-token scoring and top-k KV selection on one GPU.
 *
 * C ABI of libkvsel.so.  Every pointer argument is caller-owned; device
 * pointers are marked [device], host pointers [host].  No call allocates or
 * frees device memory and no call synchronises a stream except
 * kvsel_read_device_error() and kvsel_trace_read().  Calls are asynchronous
 * on the stream passed in; the library keeps no per-call state, so calls with
 * distinct workspaces may run concurrently from several host threads.
 *
 * Stream capture.  The calls of a step (scoring, aggregation, selection,
 * compaction, page table, attention) enqueue only kernels and memsets on the
 * stream and read host arguments at call time, so a step can be captured into
 * a CUDA graph (in any capture mode) and replayed; a replay reads the device
 * buffers as they are then, with the host arguments of the captured call.
 * kvsel_read_device_error() and kvsel_trace_read() synchronise and are not
 * for capture.
 *
 * Arguments are checked on the host before any launch; a rejected call
 * returns a status and launches nothing.  A launch failure returns
 * KVSEL_ERR_CUDA.  Errors that only the device can see (a bounded wait that
 * ran out, an index out of range, a device-resident length out of range) are
 * recorded in an error word at the start of the workspace and read back with
 * kvsel_read_device_error().
 *
 * Prefix lengths on the device.  A caller whose ragged lengths live in device
 * memory (CompactAttention, 'Future directions': page-table metadata built on
 * the kernel side, with no CPU-GPU synchronisation) sets
 * kvsel_desc.prefix_lens_dev and prefix_len_max instead of prefix_lens.  Each
 * call then builds its per-sequence offsets on the device (one small kernel
 * per call, on the call's stream) and sizes its grids for prefix_len_max.
 * What changes for the caller:
 *   - the layouts stay packed by the real lengths, but every buffer must have
 *     room for every sequence at prefix_len_max (the kernels' tensor maps and
 *     grids are sized for the bound);
 *   - every call needs a workspace, including kvsel_compact,
 *     kvsel_compact_layers and kvsel_prefill_attention;
 *   - checks that depend on a length (1 <= L_b <= prefix_len_max; kvsel_topk's
 *     k <= L_b and its page rules; kvsel_pagetable's n_kvblk, then read from
 *     device memory) run on the device: a failed check records
 *     KVSEL_ERR_INVALID_ARG (detail: the sequence) in the error word and that
 *     call's kernels leave their outputs unwritten.
 *
 * Layouts (bf16 = IEEE bfloat16 bit pattern in uint16 storage, row-major,
 * sequences of a batch packed one after another in batch order):
 *   q            [batch][n_layers][h_q][W][d]                     bf16
 *   k, v         per sequence b: [n_layers][h_kv][L_b + W][d]     bf16
 *   scores       per sequence b: [n_layers][h_kv][L_b]            fp32
 *   page_scores  per sequence b: [n_layers][h_kv][ceil(L_b / P)]  fp32
 * Key row t of sequence b is absolute prompt position t: rows 0..L_b-1 are
 * the prefix, rows L_b..L_b+W-1 the observation window whose queries are q.
 * Query head h reads KV head g = h / (h_q / h_kv).
 */
#ifndef KVSEL_H
#define KVSEL_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#if defined(__GNUC__)
#define KVSEL_API __attribute__((visibility("default")))
#else
#define KVSEL_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  KVSEL_OK = 0,
  KVSEL_ERR_INVALID_ARG = 1,   /* null pointer, bad size, inconsistent shape */
  KVSEL_ERR_UNSUPPORTED = 2,   /* valid request outside what the kernels implement */
  KVSEL_ERR_WORKSPACE = 3,     /* workspace null, misaligned or smaller than kvsel_workspace_size() */
  KVSEL_ERR_CUDA = 4,          /* a CUDA runtime call or kernel launch failed */
  KVSEL_ERR_TIMEOUT = 5,       /* a bounded device-side wait gave up */
  KVSEL_ERR_DEVICE = 6         /* the device found an index out of range */
} kvsel_status;

/* group_reduce / page_reduce: sum, max, or (group_reduce only) the mean over the G * W rows of a group */
enum { KVSEL_REDUCE_SUM = 0, KVSEL_REDUCE_MAX = 1, KVSEL_REDUCE_MEAN = 2 };
/* pool_type: max-pooling or average pooling (the mean over the in-range neighbours) */
enum { KVSEL_POOL_MAX = 0, KVSEL_POOL_AVG = 1 };
/* score_mode: post-softmax window probabilities, or the pre-softmax scaled logits */
enum { KVSEL_SCORE_SOFTMAX = 0, KVSEL_SCORE_LOGITS = 1 };
/* kvsel_aggregate: what happens across layers and across KV heads */
enum { KVSEL_LAYERS_EACH = 0, KVSEL_LAYERS_L1_MEAN = 1, KVSEL_LAYERS_MAX = 2 };
enum { KVSEL_HEADS_EACH = 0, KVSEL_HEADS_SUM = 1 };

#define KVSEL_MAX_BATCH 128
#define KVSEL_MAX_WINDOW 64
#define KVSEL_MAX_ROWS 256          /* (h_q / h_kv) * window */
#define KVSEL_MAX_PAGE 256
#define KVSEL_WS_ALIGN 256          /* required workspace alignment in bytes */

/* Shape and reduction modes shared by every call. */
typedef struct {
  int32_t n_layers;            /* >= 1 */
  int32_t h_q;                 /* query heads, multiple of h_kv */
  int32_t h_kv;                /* KV heads >= 1 */
  int32_t head_dim;            /* d: 64 or 128 */
  int32_t window;              /* W: 1 .. KVSEL_MAX_WINDOW; (h_q / h_kv) * W <= KVSEL_MAX_ROWS */
  int32_t batch;               /* sequences: 1 .. KVSEL_MAX_BATCH */
  const int64_t* prefix_lens;  /* [host] [batch] prefix lengths L_b >= 1, L_b + W < 2^31; or NULL with
                                  prefix_lens_dev */
  int32_t group_reduce;        /* KVSEL_REDUCE_SUM, _MAX or _MEAN over the query heads of a group */
  int32_t pool_k;              /* odd pool width, 1 (none) .. 63 */
  int32_t page_size;           /* P: 1 = token mode, 2 .. KVSEL_MAX_PAGE = page mode */
  int32_t page_reduce;         /* KVSEL_REDUCE_MAX or KVSEL_REDUCE_SUM over the tokens of a page */
  int32_t pool_type;           /* KVSEL_POOL_MAX (0) or KVSEL_POOL_AVG */
  int32_t score_mode;          /* KVSEL_SCORE_SOFTMAX (0) or KVSEL_SCORE_LOGITS */
  const int64_t* prefix_lens_dev;  /* [device] [batch] prefix lengths, or NULL (prefix_lens is used);
                                      exactly one of prefix_lens / prefix_lens_dev is set */
  int64_t prefix_len_max;      /* with prefix_lens_dev: bound of every L_b (>= 1, + W < 2^31); sizes the
                                  workspace, the grids and the buffers the caller provides */
} kvsel_desc;

/* Bytes of device workspace the calls below need for this descriptor (any of them). */
KVSEL_API kvsel_status kvsel_workspace_size(const kvsel_desc* desc, size_t* bytes);

/*
 * kvsel_score — window-query attention scores of every prefix token.
 *
 * ClusterAttn: KV Cache Compression under Intrinsic Attention Clustering,
 * 'Background and key observations', feature aggregation: the W window
 * queries attend to all prompt keys through a causal mask inside the window
 * (row j sees prefix keys and window keys 0..j), QK^T / sqrt(d), softmax over
 * the full row, then the post-softmax mass is summed over the window rows for
 * each prefix column.  The per-head column mass is reduced over the query
 * heads of each GQA group (sum as in CLAA's FastKV-style window scoring,
 * max as in DELTA's head-aware scoring, or the mean over the group's rows as
 * LookaheadKV averages its lookahead rows), pooled with width pool_k over
 * prefix positions (CLAA, 'Oracle construction': 1-D pooling, kernel 7; max
 * or average, out-of-range neighbours ignored), and, in page mode, reduced to
 * page scores over P consecutive tokens (DELTA, 'Key designs' 2 and 3).
 * With score_mode KVSEL_SCORE_LOGITS the softmax is skipped and the scaled
 * logits are summed instead (CLAA, 'Three representative token-ranking
 * methods': GemFilter's pre-softmax score of the last prompt token, W = 1);
 * that mode makes one pass over K instead of two.
 *
 *   q, k         [device] bf16, layouts above; 16-byte aligned
 *   scores       [device] fp32 out: pooled token scores (raw group scores when pool_k == 1)
 *   page_scores  [device] fp32 out in page mode (may be NULL in token mode)
 *   ws           [device] workspace of ws_bytes >= kvsel_workspace_size(), KVSEL_WS_ALIGN aligned
 */
KVSEL_API kvsel_status kvsel_score(const kvsel_desc* desc, const void* q, const void* k,
                         float* scores, float* page_scores,
                         void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * kvsel_prefill_attention — causal attention of every prompt row, with what the window scoring needs.
 *
 * o_i = sum over keys t <= i of softmax(q_i k_t / sqrt(d)) v_t for every row i of every query head
 * (GQA map h -> h / (h_q / h_kv)), on the tensor cores.  CLAA, 'Complete flow and cost' (engineering
 * detail 1): the keys that score the observation window are the prefill's own; the prefill's softmax
 * forms each row's log-sum-exp, which is the first of the scoring's two passes for the window rows.
 * So the call also writes the window rows' lse (base 2, units of z log2(e) / sqrt(d), in the order
 * kvsel_score_from_lse reads) and the window queries; kvsel_score_from_lse then scores with one pass.
 *
 *   q, o     [device] bf16, per sequence b: [n_layers][h_q][L_b + W][d]; d = 128
 *   k, v     [device] bf16 caches, layout above
 *   lse      [device] fp32 out, natural-log lse of every row, layout of q without d (nullable)
 *   lse_win  [device] fp32 out [batch][n_layers][h_kv][(h_q / h_kv) * W], row (h_local, j)
 *   q_win    [device] bf16 out [batch][n_layers][h_q][W][d] (the layout kvsel_score reads)
 *   ws       [device] workspace or NULL (error word for bounded waits)
 */
KVSEL_API kvsel_status kvsel_prefill_attention(const kvsel_desc* desc, const void* q, const void* k, const void* v,
                                               void* o, float* lse, float* lse_win, void* q_win, void* ws,
                                               cudaStream_t stream);

/*
 * kvsel_score_from_lse — kvsel_score with the window rows' lse given (from kvsel_prefill_attention).
 *
 * Computes what kvsel_score computes (softmax mode) with the second pass only: the column mass of
 * the window probabilities 2^(z log2(e) / sqrt(d) - lse) for every prefix key, the group reduce,
 * pooling and page reduce.  One read of the prefix keys instead of two.
 *
 *   q_win    [device] bf16 window queries, layout above
 *   lse_win  [device] fp32, as kvsel_prefill_attention writes it
 *   other arguments as for kvsel_score
 */
KVSEL_API kvsel_status kvsel_score_from_lse(const kvsel_desc* desc, const void* q_win, const void* k,
                                            const float* lse_win, float* scores, float* page_scores, void* ws,
                                            size_t ws_bytes, cudaStream_t stream);

/*
 * kvsel_combine_layers — cross-layer aggregation of raw group scores.
 *
 * Each layer's scores of a (sequence, KV head) row are L1-normalised over the
 * prefix (LookaheadKV, 'KL divergence and ListNet': s / ||s||_1), the mean is
 * taken over layers layer_lo..layer_hi inclusive (CLAA, decision 3: one score
 * per token aggregated over several layers), and the result is pooled with
 * desc->pool_k / desc->pool_type.  Same as kvsel_aggregate with
 * KVSEL_LAYERS_L1_MEAN and KVSEL_HEADS_EACH.
 *
 *   scores    [device] fp32 raw group scores (kvsel_score with pool_k = 1), layout above
 *   combined  [device] fp32 out, per sequence b: [h_kv][L_b]
 *   ws        [device] workspace (holds the per-layer L1 norms)
 */
KVSEL_API kvsel_status kvsel_combine_layers(const kvsel_desc* desc, const float* scores,
                                  int32_t layer_lo, int32_t layer_hi, float* combined,
                                  void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * kvsel_aggregate — reduce raw group scores across KV heads and layers, then pool.
 *
 * For each sequence, over layers layer_lo..layer_hi (inclusive) of raw group
 * scores (kvsel_score with pool_k = 1):
 *   head_op  KVSEL_HEADS_EACH keeps every KV head; KVSEL_HEADS_SUM sums all KV
 *            heads of a layer (the sum over all attention heads that FastKV,
 *            CLAA and GemFilter rank with; CLAA, decision 2);
 *   layer_op KVSEL_LAYERS_EACH keeps every layer of the range;
 *            KVSEL_LAYERS_L1_MEAN L1-normalises each layer's row over the prefix
 *            (LookaheadKV, 'KL divergence and ListNet') and averages the range;
 *            KVSEL_LAYERS_MAX takes the token-wise max over the range (CLAA,
 *            decision 3, Eq. 6, at the pruning layer);
 * then pools with desc->pool_k / desc->pool_type.  Token scores only.
 *
 *   scores  [device] fp32 raw group scores, per sequence b: [n_layers][h_kv][L_b]
 *   out     [device] fp32, per sequence b: [n_l][n_h][L_b], n_l = layer_hi - layer_lo + 1
 *           (EACH) or 1, n_h = h_kv (EACH) or 1; sequences packed in batch order
 *   ws      [device] workspace (holds the L1 norms)
 */
KVSEL_API kvsel_status kvsel_aggregate(const kvsel_desc* desc, const float* scores, int32_t layer_lo,
                                       int32_t layer_hi, int32_t layer_op, int32_t head_op, float* out,
                                       void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * kvsel_select — top-k selection over any rows of scores, ties to the lower index.
 *
 * As kvsel_topk (below), over `rows` score rows per sequence: per sequence b,
 * scores [rows][n] with n = L_b (token mode) or ceil(L_b / P) (page mode),
 * sequences packed in batch order.  With append_window == 0 the window
 * positions (or window pages) are not appended — for windows whose keys are
 * not part of the prompt to keep, such as LookaheadKV's lookahead rows,
 * which take no part in decoding ('Method steps').
 *
 *   idx_out  [device] int32 out [batch][rows][n_sel], n_sel = k (+ W with the
 *            window, token mode) or k + n_recent (+ W / P with the window, page mode)
 */
KVSEL_API kvsel_status kvsel_select(const kvsel_desc* desc, const float* scores, int32_t rows, int32_t k,
                                    int32_t n_recent, int32_t append_window, int32_t* idx_out,
                                    void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * kvsel_topk — top-k selection per (sequence, layer, KV head) row, ties to the lower index.
 *
 * Token mode (desc->page_size == 1): the k prefix tokens of highest score,
 * in ascending position, then the window positions L_b .. L_b+W-1 (ClusterAttn,
 * 'Method details': the compressed prefix is joined with the window).
 * Page mode: the last n_recent prefix pages are kept and the k highest-scoring
 * of the other prefix pages are added (DELTA, 'Key designs' 2: recency pages
 * union top pages of the rest), in ascending order, then the W / P pages of
 * the window.  Page mode requires W % P == 0, and n_recent >= 1 when
 * L_b % P != 0 (so the page shared by prefix and window is kept once).
 *
 *   scores   [device] fp32 per sequence b: [layers][h_kv][n] with n = L_b (token mode)
 *            or ceil(L_b / P) (page mode); layers = desc->n_layers, or 1 for the
 *            output of kvsel_combine_layers
 *   idx_out  [device] int32 out [batch][layers][h_kv][n_sel], n_sel = k + W (token)
 *            or k + n_recent + W / P (page): token positions or page numbers
 */
KVSEL_API kvsel_status kvsel_topk(const kvsel_desc* desc, const float* scores, int32_t layers,
                        int32_t k, int32_t n_recent, int32_t* idx_out,
                        void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * kvsel_compact — gather the kept K and V rows into a compacted cache.
 *
 * CLAA, 'Complete flow and cost': each layer's cache keeps only the K and V
 * rows of the selected tokens; ClusterAttn, 'Method details', keeps the window
 * rows with them.  Token mode copies row idx[r]; page mode copies the P rows
 * of page idx[r] (rows past L_b + W are written as zero).  A bit copy:
 * outputs equal inputs exactly.
 *
 *   k, v          [device] bf16 caches, layout above; either may instead be pinned
 *                 host memory mapped at the same address (cudaHostAlloc, or
 *                 cudaHostRegister with cudaHostRegisterMapped): the kernel then
 *                 reads only the kept rows over the host link, so a cache held on
 *                 the host never has to be copied whole.  Any other pointer (pageable
 *                 host memory, another device's memory) is rejected with
 *                 KVSEL_ERR_INVALID_ARG before the launch.
 *   idx           [device] int32 [batch][idx_layers][h_kv][n_sel] as written by kvsel_topk;
 *                 idx_layers == 1 applies one selection to every layer
 *   k_out, v_out  [device] bf16 out [batch][n_layers][h_kv][n_sel * P][d]
 *   ws            [device] workspace or NULL; an index out of range is not
 *                 followed, its row is zeroed and, with ws, KVSEL_ERR_DEVICE is
 *                 recorded in the error word
 */
KVSEL_API kvsel_status kvsel_compact(const kvsel_desc* desc, const void* k, const void* v,
                           const int32_t* idx, int32_t idx_layers, int32_t n_sel,
                           void* k_out, void* v_out, void* ws, cudaStream_t stream);

/*
 * kvsel_compact_layers — kvsel_compact over a range of layers, with selections shared by heads.
 *
 * Compacts layers layer_lo .. layer_lo + n_layers_out - 1 of the caches (CLAA,
 * 'Three design decisions', decision 1: the first m layers keep their full
 * cache and are not compacted).  idx is [batch][idx_layers][idx_heads][n_sel]:
 * idx_layers == 1 applies one selection to every compacted layer, otherwise
 * idx_layers == n_layers_out and row i serves layer layer_lo + i; idx_heads == 1
 * applies one selection to every KV head (the all-head scores of CLAA,
 * FastKV and GemFilter rank tokens once per layer), otherwise idx_heads == h_kv.
 *
 *   k, v          as for kvsel_compact (device, or mapped pinned host memory)
 *   k_out, v_out  [device] bf16 out [batch][n_layers_out][h_kv][n_sel * P][d]
 *   ws            [device] workspace or NULL (errors as for kvsel_compact)
 */
KVSEL_API kvsel_status kvsel_compact_layers(const kvsel_desc* desc, const void* k, const void* v,
                                            const int32_t* idx, int32_t idx_layers, int32_t idx_heads,
                                            int32_t layer_lo, int32_t n_layers_out, int32_t n_sel,
                                            void* k_out, void* v_out, void* ws, cudaStream_t stream);

/*
 * kvsel_attend — attention of a few query rows per head over the KV rows a table selects, in place.
 *
 * CompactAttention, 'Method steps' (3): the per-group block list T[b,g] (kv_indptr / kv_indices,
 * as kvsel_pagetable writes it) goes to a paged dense-attention kernel that reads the selected
 * blocks of the KV-head-major cache where they are, with no copy; DELTA, 'Overall framework':
 * sparse layers attend only over the selected page set (the dense page table of kvsel_topk in page
 * mode).  For each table row (b, layer, g) and each of the n_q query rows of each of the G query
 * heads of group g: o = softmax(q K_sel^T / sqrt(d)) V_sel over every row of every listed block
 * (block j covers rows j*block .. j*block + block - 1; rows past L_b + W do not exist), with no
 * causal mask (decode-style queries come after every selected key).  A row that selects nothing
 * gives o = 0.
 *
 *   q           [device] bf16 [batch][n_layers][h_q][n_q][d]; (h_q / h_kv) * n_q <= 32
 *   k, v        [device] bf16 caches, layout above
 *   kv_indptr   [device] int32 [batch * n_layers * h_kv + 1] (CSR), or NULL: row r's list is
 *               kv_indices[r * n_per_row .. (r + 1) * n_per_row) (a dense table)
 *   kv_indices  [device] int32 block ids, or NULL together with kv_indptr: every block of the
 *               row's cache in order (dense attention over the whole cache)
 *   block       rows per block, 1 .. KVSEL_MAX_PAGE
 *   max_blocks  upper bound of any row's list length (sizes the split of each row's work)
 *   o           [device] fp32 out [batch][n_layers][h_q][n_q][d]
 *   ws          [device] workspace of kvsel_attend_workspace_size() bytes (partials of the splits);
 *               a block id whose first row does not exist is skipped and KVSEL_ERR_DEVICE recorded.
 *               The split count, and with it the size, depends on how many warps the current device
 *               keeps resident: query the size on the device the call runs on.
 *
 * Arithmetic: for up to 8 query rows per table row the logits are bf16 products accumulated in fp32
 * (tensor cores) and P V takes P to ~16 significant bits (a bf16 high and low part); more rows use
 * fp32 FMA throughout.
 */
KVSEL_API kvsel_status kvsel_attend_workspace_size(const kvsel_desc* desc, int32_t n_q, int32_t block,
                                                   int32_t max_blocks, size_t* bytes);
KVSEL_API kvsel_status kvsel_attend(const kvsel_desc* desc, const void* q, int32_t n_q, const void* k,
                                    const void* v, const int32_t* kv_indptr, const int32_t* kv_indices,
                                    int32_t n_per_row, int32_t block, int32_t max_blocks, float* o, void* ws,
                                    size_t ws_bytes, cudaStream_t stream);

/*
 * kvsel_claa_shape / kvsel_claa_select — the CLAA schedule over one prompt.
 *
 * CLAA, 'Three design decisions': decision 1, the first m layers (defer) keep their full cache;
 * decision 2, every later layer up to the pruning layer l_p scores the prompt with its observation
 * window (post-softmax probabilities summed over the window rows and all heads); decision 3 (Eq. 6),
 * the per-layer scores of the last n layers (the rolling buffer, layers max(m, l_p - n + 1) .. l_p)
 * are aggregated token-wise by their maximum.  'Complete flow and cost': each scored layer keeps
 * topk(score, keep_rate) of the prefix (k = floor(r L + 1/2), clipped to [0, L]) plus the window and
 * gathers its cache to those rows; at l_p the pooled aggregate picks the sequence prune index.
 * Pooling is desc->pool_k / pool_type ('Experimental setup': average pooling, kernel 7).
 *
 * The descriptor covers every layer of the prompt (batch 1, host prefix length, token mode,
 * group_reduce KVSEL_REDUCE_SUM, score_mode KVSEL_SCORE_SOFTMAX).  kvsel_claa_shape returns the
 * sizes the outputs need; kvsel_claa_select runs the schedule:
 *   q, k, v        [device] bf16, layouts above, all n_layers layers; v is only gathered, so it
 *                  may be mapped pinned host memory (as for kvsel_compact)
 *   scores         [device] fp32 out [n_scored][h_kv][L]: raw group scores of layers m .. l_p
 *   layer_scores   [device] fp32 out [n_scored][L]: pooled all-head score of each scored layer
 *   prune_scores   [device] fp32 out [L]: pooled token-wise max over the buffer
 *   idx            [device] int32 out [n_scored][n_sel]: each scored layer's kept rows
 *   prune_idx      [device] int32 out [n_sel]: the prune index
 *   k_out, v_out   [device] bf16 out [n_scored][h_kv][n_sel][d]: compacted caches of layers m .. l_p
 *   ws             [device] workspace of at least shape.ws_bytes
 */
typedef struct {
  int32_t defer;          /* m: layers 0 .. m - 1 are neither scored nor compacted */
  int32_t prune_layer;    /* l_p: m <= l_p < n_layers */
  int32_t n_buffer;       /* n >= 1: layers in the rolling buffer */
  double keep_rate;       /* r in [0, 1]: fraction of the prefix kept */
} kvsel_claa_params;

typedef struct {
  int32_t n_scored;       /* l_p - m + 1 */
  int32_t buffer_lo;      /* first buffered layer, max(m, l_p - n + 1); the last is l_p */
  int32_t k;              /* prefix tokens kept per selection */
  int32_t n_sel;          /* entries per selection: k + W */
  size_t ws_bytes;        /* workspace kvsel_claa_select needs */
} kvsel_claa_shape_t;

KVSEL_API kvsel_status kvsel_claa_shape(const kvsel_desc* desc, const kvsel_claa_params* p, kvsel_claa_shape_t* out);
KVSEL_API kvsel_status kvsel_claa_select(const kvsel_desc* desc, const kvsel_claa_params* p, const void* q,
                                         const void* k, const void* v, float* scores, float* layer_scores,
                                         float* prune_scores, int32_t* idx, int32_t* prune_idx, void* k_out,
                                         void* v_out, void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * kvsel_pagetable — per-group KV block table from a 2-D block mask.
 *
 * CompactAttention: Accelerating Chunked Prefill with Block-Union KV
 * Selection, 'Method steps' (2): Q-block union Mbar[b,h,j] = OR_i M[b,h,i,j],
 * intra-group union G[b,g,j] = OR over the heads h of group g, and
 * T[b,g] = { j : G[b,g,j] = 1 } in ascending order, written as CSR
 * (kv_indptr / kv_indices) over rows (b, layer, g).
 *
 *   mask        [device] uint8 [batch][n_layers][h_q][n_qblk][n_kvblk_max], nonzero = selected
 *   n_kvblk     [host] [batch] KV blocks of each sequence (<= n_kvblk_max); mask
 *               entries at j >= n_kvblk[b] are ignored.  [device] when the descriptor's
 *               prefix lengths are on the device (prefix_lens_dev)
 *   kv_indptr   [device] int32 out [batch * n_layers * h_kv + 1]
 *   kv_indices  [device] int32 out, capacity batch * n_layers * h_kv * n_kvblk_max
 */
KVSEL_API kvsel_status kvsel_pagetable(const kvsel_desc* desc, const uint8_t* mask, int32_t n_qblk,
                             int32_t n_kvblk_max, const int32_t* n_kvblk,
                             int32_t* kv_indptr, int32_t* kv_indices,
                             void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * Decoding on over a paged cache.
 *
 * The calls above score, select and compact a prompt's cache, which is packed and of fixed size.  The
 * calls below carry the decode that follows: a pool of pages holds the rows of many requests, each
 * request lists its pages in a block table, and a step of one or more new rows per request runs
 *   kvsel_page_assign   pages, slots and positions of the step's new rows (once for all layers),
 *   kvsel_rope_append   norm, rotation and the write of the new K / V rows (per layer),
 *   kvsel_paged_attend  attention of one new query row per head over the request's rows (per layer).
 * Lengths, tables and slots live in device memory and nothing synchronises, so a step can be captured.
 * DELTA, 'Key designs' 3 (caches in pages of P tokens); CompactAttention, 'Future directions' (page
 * metadata built on the kernel side, without a CPU-GPU synchronisation).
 *
 * Row t of a request is row t % P of page block_table[t / P]; its slot is page * P + t % P.
 */
enum { KVSEL_DTYPE_BF16 = 0, KVSEL_DTYPE_F16 = 1, KVSEL_DTYPE_E4M3 = 2, KVSEL_DTYPE_F32 = 3 };   /* F32: logits alone */

#define KVSEL_PAGED_MAX_BATCH 4096

/* A pool of pages of one layer's K (and one of its V): the row of KV head g at slot s starts at element
 * (s / P) * page_stride + g * head_stride + (s % P) * row_stride and is contiguous.  Both orders of a page
 * (heads outside rows, rows outside heads) are strides, and so is a packed [h_kv][rows][d] cache.
 * Every row of every page is memory that a call may read, whatever it holds. */
typedef struct {
  int32_t h_q;            /* query heads, multiple of h_kv */
  int32_t h_kv;           /* KV heads >= 1 */
  int32_t head_dim;       /* d: a multiple of 16, 16 .. 256 (kvsel_paged_attend: 64 or 128) */
  int32_t page_size;      /* P: rows per page, 1 .. KVSEL_MAX_PAGE */
  int64_t n_pages;        /* pages of the pool: 1 .. 2^31 - 1 */
  int32_t dtype;          /* q, k, v, weights and outputs: KVSEL_DTYPE_BF16 or KVSEL_DTYPE_F16 */
  int32_t cache_dtype;    /* the pool: dtype, or KVSEL_DTYPE_E4M3 (a value times its head's scale) */
  int64_t page_stride;    /* in elements of the pool; each a multiple of 16 bytes and >= 0 */
  int64_t head_stride;
  int64_t row_stride;
} kvsel_cache_desc;

/*
 * kvsel_page_assign — pages, slots, positions and block tables of a step's new rows, from lengths.
 *
 * Request b holds lens[b] rows (in its first ceil(lens[b] / P) table entries) and gets n_new[b] more.
 * The pages it lacks are taken from the queue free_pages[free_head ..) in request order and written to
 * its table behind the ones it has; every other table entry is left as it was.  The step's tokens are
 * numbered request by request: token indptr[b] + i is row t = lens[b] + i of request b, with
 *   slots      = table[t / P] * P + t % P
 *   positions  = t + pos_offset[b]      (a compacted cache holds fewer rows than its text has positions)
 *   seq_ids    = b
 * Tokens from indptr[batch] to max_tokens (the padding of a captured step) get slot -1, position 0 and
 * request -1.  The updated lengths and queue head may be written over the old ones, so that the replays
 * of a captured step go on from one another.
 *
 *   lens, n_new    [device] int64 [batch]
 *   pos_offset     [device] int64 [batch], or NULL (0)
 *   free_pages     [device] int32 [n_free] page ids, each in [0, n_pages)
 *   free_head      [device] int64 [1]: entries of free_pages taken so far
 *   block_tables   [device] int32 [batch][max_blocks], in and out
 *   lens_out       [device] int64 [batch] out: lens + n_new; may be lens
 *   free_head_out  [device] int64 [1] out; may be free_head
 *   indptr         [device] int64 [batch + 1] out
 *   slots          [device] int64 [max_tokens] out
 *   positions      [device] int64 [max_tokens] out (nullable)
 *   seq_ids        [device] int32 [max_tokens] out (nullable)
 *   ws             [device] workspace of kvsel_page_assign_workspace_size() bytes
 *
 * A step that cannot be carried out (a negative length or count, a request longer than max_blocks * P
 * rows, more than max_tokens tokens, a queue with too few pages or a head outside it) records
 * KVSEL_ERR_INVALID_ARG (detail: the request, or batch for the sums) and assigns nothing: slots -1,
 * positions 0, requests -1, indptr 0, lengths and head unchanged, tables as they were.  A page id outside
 * [0, n_pages) records KVSEL_ERR_DEVICE and its rows get slot -1.
 */
KVSEL_API kvsel_status kvsel_page_assign_workspace_size(int32_t batch, size_t* bytes);
KVSEL_API kvsel_status kvsel_page_assign(int32_t page_size, int64_t n_pages, int32_t batch, int32_t max_blocks,
                                         const int64_t* lens, const int64_t* n_new, const int64_t* pos_offset,
                                         const int32_t* free_pages, int64_t n_free, const int64_t* free_head,
                                         int32_t* block_tables, int64_t* lens_out, int64_t* free_head_out,
                                         int64_t* indptr, int64_t max_tokens, int64_t* slots, int64_t* positions,
                                         int32_t* seq_ids, void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * kvsel_rope_freqs — angles per position of rotary pairs, with the long-context scalings.  Host only.
 *
 * theta_i = base^(-2 i / rot_dim), i < rot_dim / 2, then
 *   PLAIN   theta
 *   LINEAR  theta / factor
 *   BANDED  by the pair's wavelength w = 2 pi / theta against the original context L0: theta where
 *           w < L0 / high, theta / factor where w > L0 / low, between them
 *           (1 - s) theta / factor + s theta with s = (L0 / w - low) / (high - low)
 *   RAMP    by the pair's index: r theta / factor + (1 - r) theta with r rising linearly from 0 to 1
 *           between the (whole) indexes whose pairs turn `high` and `low` times over L0; cos and sin are
 *           scaled by 0.1 ln(factor) + 1
 *
 *   inv_freq  [host] double [rot_dim / 2] out: radians per position (kvsel_rope_append reads it from
 *             device memory)
 *   scale     [host] float out: the factor on cos and sin (kvsel_rope_desc.factor)
 */
enum { KVSEL_ROPE_PLAIN = 0, KVSEL_ROPE_LINEAR = 1, KVSEL_ROPE_BANDED = 2, KVSEL_ROPE_RAMP = 3 };
typedef struct {
  int32_t type;           /* KVSEL_ROPE_PLAIN .. KVSEL_ROPE_RAMP */
  double base;            /* > 1 */
  double factor;          /* >= 1 (not read by PLAIN) */
  double low, high;       /* BANDED, RAMP: 0 < low < high */
  int64_t original_len;   /* BANDED, RAMP: L0 >= 1 */
} kvsel_rope_scaling;
KVSEL_API kvsel_status kvsel_rope_freqs(int32_t rot_dim, const kvsel_rope_scaling* scaling, double* inv_freq,
                                        float* scale);

/*
 * kvsel_rope_append — norm and rotation of the new queries and keys, and the new K / V rows into the pool.
 *
 * For every token i with slots[i] >= 0 and every head of q and k:
 *   y = x / sqrt(mean(x^2) + norm_eps) * (weight + weight_bias)     (with a weight; else y = x)
 *   the pairs of the first rot_dim elements of y turn by positions[i] * inv_freq[pair]:
 *   (a, b) -> factor * (a cos - b sin, b cos + a sin); HALF pairs element j with j + rot_dim / 2,
 *   INTERLEAVED 2 j with 2 j + 1; the other elements pass.
 * q goes to q_out, k and v (v as it is) to the rows of `slots` in the pools; in an e4m3 pool value x is held
 * as x / scale of its head, rounded to nearest and clamped to +-448.  Tokens with slot -1 are padding:
 * nothing of theirs is written.  All arithmetic is fp32 with one rounding at the end; angles are formed
 * to 2^-32 of a turn at any frequency below 2^50 and position below 2^31, their cosines and sines to 2^-22.
 * No tokens (n_tokens 0): nothing to do, whatever the pointers.
 *
 *   q          [device] dtype, element (i, h, c) at i * q_stride + h * q_head_stride + c; NULL with q_out:
 *              keys and values only (rows of a compacted cache: rot_dim 0, no weights)
 *   k, v       [device] dtype, likewise; NULL together with the pools: queries only
 *   positions  [device] int64 [n_tokens]; inv_freq [device] double [rot_dim / 2]; both NULL with rot_dim 0
 *   slots      [device] int64 [n_tokens]; may be NULL when k and v are (no token is padding)
 *   q_weight, k_weight  [device] dtype [d], or NULL: no norm
 *   q_out      [device] dtype [n_tokens][h_q][d]; may be q when q is laid out the same
 *   k_cache, v_cache  [device] pools; the slots of a call are distinct (a slot named twice holds one of the
 *              rows, or parts of both)
 *   k_scale, v_scale  [device] fp32 [h_kv], both given exactly when the pool is e4m3
 *   ws         [device] workspace or NULL (the error word): a slot outside [-1, n_pages * P) is not written
 *              and, with ws, KVSEL_ERR_DEVICE is recorded (detail: the token)
 */
enum { KVSEL_ROPE_HALF = 0, KVSEL_ROPE_INTERLEAVED = 1 };
typedef struct {
  int32_t rot_dim;        /* 0 (no rotation) .. d, a multiple of 16 */
  int32_t layout;         /* KVSEL_ROPE_HALF or KVSEL_ROPE_INTERLEAVED */
  float factor;           /* on cos and sin */
  float norm_eps;         /* >= 0 */
  float weight_bias;      /* added to the norm weights (0, or 1 for weights stored as w - 1) */
  int64_t q_stride, q_head_stride;   /* elements, each a multiple of 8 (16 bytes) */
  int64_t k_stride, k_head_stride;
  int64_t v_stride, v_head_stride;
} kvsel_rope_desc;
KVSEL_API kvsel_status kvsel_rope_append(const kvsel_cache_desc* cache, const kvsel_rope_desc* rope, int64_t n_tokens,
                                         const void* q, const void* k, const void* v, const int64_t* positions,
                                         const int64_t* slots, const void* q_weight, const void* k_weight,
                                         const double* inv_freq, void* q_out, void* k_cache, void* v_cache,
                                         const float* k_scale, const float* v_scale, void* ws, cudaStream_t stream);

/*
 * kvsel_paged_attend — attention of one new query row per head over a request's rows in the pool.
 *
 * Request b with n = lens[b] rows (its newest row, the query's own, among them) sees rows
 * t in [max(0, n - window), n), or all n without a window:
 *   z_t = scale <q, k_t>;  with softcap c: z_t = c tanh(z_t / c);  with slopes: z_t += slope_h (t - (n - 1))
 *   o = sum_t softmax(z)_t v_t,  lse = log sum_t exp(z_t)
 * Query head h reads KV head h / (h_q / h_kv).  A request with no row gives o = 0 and lse = -inf.  Rows
 * that a request does not see take no part whatever the pool holds there (infinities and NaN too).
 *
 *   q             [device] dtype, element (b, h, c) at b * q_stride + h * d + c
 *   k_cache, v_cache  [device] pools
 *   block_tables  [device] int32 [batch][max_blocks]; entries behind a request's last page are not read
 *   lens          [device] int64 [batch]
 *   slopes        [device] fp32 [h_q], or NULL
 *   k_scale, v_scale  [device] fp32 [h_kv], both given exactly when the pool is e4m3
 *   o             [device] dtype [batch][h_q][d] out
 *   lse           [device] fp32 [batch][h_q] out, or NULL
 *   ws            [device] workspace of kvsel_paged_attend_workspace_size() bytes (the splits' partials);
 *                 the size depends on the current device: query it where the call runs
 *
 * A length outside [0, max_blocks * P] records KVSEL_ERR_INVALID_ARG (detail: the request), which then
 * counts as empty; a page id outside [0, n_pages) records KVSEL_ERR_DEVICE (detail: the request) and its
 * rows are left out.
 *
 * Arithmetic: products of the 16-bit values (e4m3 values as fp16, exactly) accumulated in fp32 on the
 * tensor cores, softmax statistics in fp32, P taken as a high and a low 16-bit part (2^-17 of a weight; with fp16
 * and e4m3 pools also 2^-38 of the row's largest weight).  With an e4m3 pool the query row is held in fp16
 * scaled by a power of two of its own (2^-24 of the row's largest value).
 */
typedef struct {
  int32_t batch;          /* requests: 1 .. KVSEL_PAGED_MAX_BATCH */
  int32_t max_blocks;     /* columns of the block tables >= 1, (max_blocks + 1) * P < 2^31 */
  int64_t q_stride;       /* elements between requests' queries, a multiple of 8; 0: h_q * d */
  float scale;            /* on the scores; 0: 1 / sqrt(d) */
  float softcap;          /* c in [2^-126, 2^127], or 0: none */
  int32_t window;         /* rows seen, >= 1, or 0: all */
} kvsel_paged_attend_desc;
KVSEL_API kvsel_status kvsel_paged_attend_workspace_size(const kvsel_cache_desc* cache,
                                                         const kvsel_paged_attend_desc* desc, size_t* bytes);
KVSEL_API kvsel_status kvsel_paged_attend(const kvsel_cache_desc* cache, const kvsel_paged_attend_desc* desc,
                                          const void* q, const void* k_cache, const void* v_cache,
                                          const int32_t* block_tables, const int64_t* lens, const float* slopes,
                                          const float* k_scale, const float* v_scale, void* o, float* lse, void* ws,
                                          size_t ws_bytes, cudaStream_t stream);

/*
 * kvsel_chunk_attend — attention of many new tokens of each request over its rows in the pool.
 *
 * Request b's new tokens are indptr[b] .. indptr[b + 1] - 1 of q (kvsel_page_assign's offsets), the last
 * n_b = indptr[b + 1] - indptr[b] of its lens[b] rows, whose K and V rows are in the pool already.  Token i of
 * them is row p = lens[b] - n_b + i and sees rows t in [max(0, p + 1 - window), p], or all up to p without a window:
 *   z_t = scale <q, k_t>;  with softcap c: z_t = c tanh(z_t / c);  with slopes: z_t += slope_h (t - p)
 *   o = sum_t softmax(z)_t v_t,  lse = log sum_t exp(z_t)
 * A prompt's chunk, a whole prompt and the tokens of a draft are such calls.  Query head h reads KV head
 * h / (h_q / h_kv).  Rows that a token does not see take no part in its output whatever the pool holds there
 * (infinities and NaN too), and rows of o and lse that belong to no request's tokens are left as they were.
 *
 *   q             [device] dtype, element (i, h, c) at i * q_stride + h * d + c, max_tokens rows
 *   k_cache, v_cache  [device] pools
 *   block_tables  [device] int32 [batch][max_blocks]; entries behind a request's last page are not read
 *   lens          [device] int64 [batch], the new tokens among them
 *   indptr        [device] int64 [batch + 1], rising, within [0, max_tokens]
 *   slopes        [device] fp32 [h_q], or NULL
 *   k_scale, v_scale  [device] fp32 [h_kv], both given exactly when the pool is e4m3
 *   o             [device] dtype [max_tokens][h_q][d] out; must not overlap q
 *   lse           [device] fp32 [max_tokens][h_q] out, or NULL
 *   ws            [device] workspace of kvsel_chunk_attend_workspace_size() bytes; the size depends on the
 *                 current device: query it where the call runs
 *
 * A length outside [0, max_blocks * P], offsets that fall or leave [0, max_tokens], or more new tokens than rows record
 * KVSEL_ERR_INVALID_ARG (detail: the request), whose tokens are then left as they were (where offsets fall, a later request
 * may claim tokens of an earlier one: which of the two writes them is open); a page id outside
 * [0, n_pages) records KVSEL_ERR_DEVICE (detail: the request) and its rows are left out.
 *
 * Arithmetic: products of 16-bit values (e4m3 values as fp16, exactly) accumulated in fp32 on the tensor cores, softmax
 * statistics in fp32, each weight rounded once to the products' 16-bit type: by at most 2^-8 of it over bf16, 2^-11 of it or
 * 2^-33 of the row's largest weight over fp16 products (a 16-bit value, where kvsel_paged_attend holds two).  With an e4m3
 * pool the query row is held in fp16 scaled by a power of two of its own (2^-24 of the row's largest value).
 */
typedef struct {
  int32_t batch;          /* requests: 1 .. KVSEL_PAGED_MAX_BATCH */
  int32_t max_blocks;     /* columns of the block tables >= 1, (max_blocks + 1) * P < 2^31 */
  int64_t max_tokens;     /* rows of q, o and lse: 0 .. 2^31 - 1, times h_q / h_kv below 2^31 */
  int64_t q_stride;       /* elements between tokens' queries, a multiple of 8; 0: h_q * d */
  float scale;            /* on the scores; 0: 1 / sqrt(d) */
  float softcap;          /* c in [2^-126, 2^127], or 0: none */
  int32_t window;         /* rows seen, >= 1, or 0: all */
} kvsel_chunk_attend_desc;
KVSEL_API kvsel_status kvsel_chunk_attend_workspace_size(const kvsel_cache_desc* cache,
                                                         const kvsel_chunk_attend_desc* desc, size_t* bytes);
KVSEL_API kvsel_status kvsel_chunk_attend(const kvsel_cache_desc* cache, const kvsel_chunk_attend_desc* desc,
                                          const void* q, const void* k_cache, const void* v_cache,
                                          const int32_t* block_tables, const int64_t* lens, const int64_t* indptr,
                                          const float* slopes, const float* k_scale, const float* v_scale, void* o,
                                          float* lse, void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * kvsel_prefix_attend — kvsel_paged_attend for a batch whose requests share long prefixes, each read once.
 *
 * What it computes is kvsel_paged_attend's, of the same arguments.  Requests group_indptr[j] .. group_indptr[j + 1] - 1
 * name the same pages for their first shared_lens[j] rows (beams of one prompt, requests behind one system prompt);
 * of those rows the whole pages are read once for all of them, through the first one's table, and every
 * request's other rows through its own.  A group of one request, or of no shared rows, is an ordinary request.
 *
 *   n_groups      1 .. batch
 *   group_indptr  [device] int64 [n_groups + 1], rising, from 0 to batch
 *   shared_lens   [device] int64 [n_groups]: at most the shortest length of the group
 *   others        as kvsel_paged_attend's; ws of kvsel_prefix_attend_workspace_size() bytes
 *
 * Offsets that fall or do not run from 0 to batch record KVSEL_ERR_INVALID_ARG (detail: batch) and no rows count as shared; a
 * shared length below 0 or above a member's length records it (detail: the group's first request) and the group's
 * rows count as not shared: the output is right either way.  Other errors are kvsel_paged_attend's; those of
 * a shared page name the group's first request.
 *
 * Arithmetic: kvsel_paged_attend's, the shared rows' and the own rows' parts joined in fp32; but with an e4m3 pool a
 * shared row's weight is rounded once to fp16 (by at most 2^-11 of it, or 2^-38 of the row's largest) instead of held in two
 * parts.
 */
KVSEL_API kvsel_status kvsel_prefix_attend_workspace_size(const kvsel_cache_desc* cache,
                                                          const kvsel_paged_attend_desc* desc, int32_t n_groups,
                                                          size_t* bytes);
KVSEL_API kvsel_status kvsel_prefix_attend(const kvsel_cache_desc* cache, const kvsel_paged_attend_desc* desc,
                                           int32_t n_groups, const void* q, const void* k_cache, const void* v_cache,
                                           const int32_t* block_tables, const int64_t* lens,
                                           const int64_t* group_indptr, const int64_t* shared_lens,
                                           const float* slopes, const float* k_scale, const float* v_scale, void* o,
                                           float* lse, void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * kvsel_beam_select — the best continuations of every set of beams.
 *
 * With x the logits of beam k of a set and s_k the sum of log probabilities it has so far,
 *   score(k, v) = s_k + x_v - log sum_u exp(x_u)
 * An ended beam has one continuation, pad_token at s_k; its other tokens are at -inf.  A set's outputs are the n_out
 * best of its beams * vocab continuations, best first; of equal scores the smaller beam first, in a beam the larger
 * logit and then the smaller token.  A NaN logit counts as -inf; scores that are no finite number (a beam at -inf, whose
 * log-sum is infinite, or whose s_k is not finite) count as -inf, and such a beam's tokens come in their order.
 *
 *   logits      [device] dtype, row batch * beams major: element (b, k, v) at (b * beams + k) * row_stride + v
 *   scores      [device] fp32 [batch][beams]
 *   ended       [device] uint8 [batch][beams], or NULL: none
 *   scores_out  [device] fp32 [batch][n_out] out; must not overlap scores
 *   parents     [device] int32 [batch][n_out] out: k
 *   tokens      [device] int32 [batch][n_out] out: v
 *   lse         [device] fp32 [batch][beams] out: log sum exp of the row, or NULL
 *   ws          [device] workspace of kvsel_beam_select_workspace_size() bytes
 *
 * Scores are formed and compared in fp64 and rounded once.  Of a log-sum, exponentials are within 2^-22 of their own (of
 * either sign, so that the sum of many is nearer); each of 256 threads adds its own in fp32, 32 of every 8192 tokens, and
 * the threads' sums are added exactly: it is within 2^-18 + 2^-21 ceil(vocab / 8192), and the same for equal rows of a call.
 */
typedef struct {
  int32_t batch;          /* sets >= 1; batch * beams at most KVSEL_PAGED_MAX_BATCH */
  int32_t beams;          /* 1 .. 64 */
  int32_t n_out;          /* 1 .. 64, at most beams * vocab */
  int32_t vocab;          /* >= 1; beams * ceil(vocab / 8192) at most 8192 */
  int32_t dtype;          /* KVSEL_DTYPE_BF16, KVSEL_DTYPE_F16 or KVSEL_DTYPE_F32 */
  int32_t pad_token;      /* in [0, vocab) */
  int64_t row_stride;     /* elements between rows, >= 0; 0: vocab */
} kvsel_beam_select_desc;
KVSEL_API kvsel_status kvsel_beam_select_workspace_size(const kvsel_beam_select_desc* desc, size_t* bytes);
KVSEL_API kvsel_status kvsel_beam_select(const kvsel_beam_select_desc* desc, const void* logits, const float* scores,
                                         const uint8_t* ended, float* scores_out, int32_t* parents, int32_t* tokens,
                                         float* lse, void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * kvsel_beam_reorder — the beams' pages after a selection.
 *
 * Set b's beams are requests b * beams .. + beams - 1 of the block tables.  Child j of a set goes on from beam
 * p = parents[b][j]: it gets p's length and names p's pages.  Pages that the set named and names no more are freed, in
 * the order (set, column, beam): put into free_pages in front of free_head.  Of the children of one parent every
 * one but the first gets its own copy of the last page if that is part full (rows 0 .. len % P - 1 of every
 * layer's K and V), in pages taken from the queue in the order (set, child), the freed ones first; so a page that is not
 * full is always one beam's alone.  All parents 0 share a prompt's pages among beams that held none.
 * Beams that share a page name it in the same column.  A page of several sets must be named by every beam of them.
 *
 *   cache             pools as in the other calls (head_dim any of its values); dtype is not looked at
 *   parents           [device] int32 [batch][beams]
 *   lens              [device] int64 [batch * beams]
 *   block_tables      [device] int32 [batch * beams][max_blocks]
 *   free_pages        [device] int32 [n_free], in and out
 *   free_head         [device] int64 [1]: entries of free_pages taken so far
 *   block_tables_out  [device] out: entries of the pages held (others are left as they were); may be block_tables
 *   lens_out          [device] out; may be lens
 *   free_head_out     [device] out; may be free_head
 *   k_cache, v_cache  [device] pools of the first layer, layer l's layer_stride * l elements on
 *   ws                [device] workspace of kvsel_beam_reorder_workspace_size() bytes
 *
 * A parent outside [0, beams), a length outside [0, max_blocks * P] (detail: the set's first request), a head outside the
 * queue or with too few entries on either side (detail: batch * beams) records KVSEL_ERR_INVALID_ARG, a page id outside
 * [0, n_pages) KVSEL_ERR_DEVICE; nothing is written then.
 */
typedef struct {
  int32_t batch;          /* sets >= 1; batch * beams at most KVSEL_PAGED_MAX_BATCH */
  int32_t beams;          /* 1 .. 64 */
  int32_t max_blocks;     /* columns of the block tables >= 1, (max_blocks + 1) * P < 2^31 */
  int32_t n_layers;       /* >= 1 */
  int64_t layer_stride;   /* elements of the pool, a multiple of 16 bytes, >= 0 */
} kvsel_beam_reorder_desc;
KVSEL_API kvsel_status kvsel_beam_reorder_workspace_size(const kvsel_beam_reorder_desc* desc, size_t* bytes);
KVSEL_API kvsel_status kvsel_beam_reorder(const kvsel_cache_desc* cache, const kvsel_beam_reorder_desc* desc,
                                          const int32_t* parents, const int64_t* lens, const int32_t* block_tables,
                                          int32_t* free_pages, int64_t n_free, const int64_t* free_head,
                                          int32_t* block_tables_out, int64_t* lens_out, int64_t* free_head_out,
                                          void* k_cache, void* v_cache, void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * kvsel_score_noalloc — kvsel_score for callers that cannot allocate device memory.
 *
 * The pages have no counterpart to this call; it exists for callers with no
 * way to obtain a workspace: a plugin inside a host program that owns all of
 * the GPU's memory, or a latency-critical caller that must not pay
 * cudaMalloc's device-wide synchronisation.  It computes exactly what
 * kvsel_score computes, with the scratch of the two scoring passes in an
 * array inside the library of KVSEL_NOALLOC_SCRATCH_BYTES, which every GPU
 * that loads the library holds until the process exits.  It allocates and
 * frees nothing.
 *
 * The first call made while a device is current looks up that array's device
 * address (cudaGetSymbolAddress) and caches it for the life of the process;
 * make that first call before any stream capture.  cudaDeviceReset after it
 * is not supported (the module may then load at another address and the
 * cached one would be stale).  The stream must belong to the current device.
 * All calls share the one array: calls whose work overlaps on the GPU (two
 * streams, or two host threads) race and give undefined results.  Arguments
 * are checked as kvsel_score checks them, and a descriptor whose
 * kvsel_workspace_size() exceeds KVSEL_NOALLOC_SCRATCH_BYTES is rejected with
 * KVSEL_ERR_WORKSPACE; a rejected call launches nothing and enqueues nothing.
 *
 * Errors only the device sees (a bounded wait that ran out) go to the error
 * word at the start of the array, which each call clears first; read it with
 * kvsel_noalloc_read_device_error() on the call's stream before the next call.
 */
#define KVSEL_NOALLOC_SCRATCH_BYTES (32u << 20)
KVSEL_API kvsel_status kvsel_score_noalloc(const kvsel_desc* desc, const void* q, const void* k,
                                           float* scores, float* page_scores, cudaStream_t stream);

/* Reads (stream-synchronising) and clears the error word of the current device's built-in scratch:
 * the status of the last kvsel_score_noalloc call on that device, or KVSEL_OK. */
KVSEL_API kvsel_status kvsel_noalloc_read_device_error(cudaStream_t stream);

/*
 * kvsel_selftest_bounded_wait — exercises the bounded device wait used by every pipelined kernel.
 *
 * The pages have no counterpart to this call; it exists so that failure reporting can be tested
 * without a real fault.  It launches one CTA that waits on a shared-memory mbarrier with the same
 * wait routine the scoring kernels use.  With arrive == 0 nothing completes the barrier, the wait
 * gives up after `polls` polls (1 .. 2^22) and KVSEL_ERR_TIMEOUT is recorded in the error word of
 * `ws` (read it with kvsel_read_device_error); with arrive != 0 a second thread completes the
 * barrier and nothing is recorded.
 */
KVSEL_API kvsel_status kvsel_selftest_bounded_wait(void* ws, uint32_t polls, int32_t arrive, cudaStream_t stream);

/* Reads (stream-synchronising) and clears the device error word of a workspace. */
KVSEL_API kvsel_status kvsel_read_device_error(void* ws, cudaStream_t stream);

KVSEL_API const char* kvsel_status_string(kvsel_status status);
KVSEL_API const char* kvsel_version(void);

/*
 * Tracing.  With tracing on, every kernel launch of the library is bracketed
 * by CUDA events on its stream; kvsel_trace_read() synchronises those events
 * and returns, per kernel name, the launches and the summed milliseconds since
 * the last read.  kvsel_launch_count() counts every kernel launch since load.
 */
typedef struct {
  char name[48];
  int64_t launches;
  double ms;
} kvsel_trace_entry;

KVSEL_API void kvsel_trace_enable(int32_t on);
KVSEL_API kvsel_status kvsel_trace_read(kvsel_trace_entry* out, int32_t capacity, int32_t* n_out);
KVSEL_API int64_t kvsel_launch_count(void);

#ifdef __cplusplus
}
#endif

#endif /* KVSEL_H */
