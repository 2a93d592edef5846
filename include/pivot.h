/*
 * pivot.h -- C ABI of the B200 (sm_100a) PIVOT query-group indexer.
 *
 * The operation is the indexer of token-level sparse attention and its PIVOT
 * replacement, as described in "PIVOT: Efficient Query-Group Indexing for
 * Token-Level Sparse Attention" (arXiv 2607.24593): the pages "PIVOT explained
 * -- from paper to working code in 10 minutes" (sections "The Problem", "How It
 * Works", "Show Me The Code") and the paper's abstract.
 *
 * Common conventions (all entry points):
 *  - Tensors are row-major, bfloat16 for q and k ("const void*" pointing to
 *    2-byte bf16 values), int32 for indices.  All tensor pointers are DEVICE
 *    pointers, 16-byte aligned.  The caller owns every buffer; the library keeps
 *    no pointer after the call returns.
 *  - Calls are asynchronous: work is enqueued on `stream` (a cudaStream_t passed
 *    as void*; NULL = the legacy default stream) and the call returns without
 *    synchronising.  Outputs are valid once the stream has reached that point.
 *  - Scores are unscaled dot products q . k.  A query at position pos may only
 *    select keys j < pos.  Ties in score go to the lower key index.  Every
 *    output row holds its selected key indices in ascending order, followed by
 *    -1 padding up to top_k.
 *  - head_dim d must be 64 or 128; 1 <= top_k <= Kc <= 4096.
 *  - Return value: PIVOT_OK, or an error code with a message available from
 *    pivot_last_error() (thread-local).  Argument errors are detected on the
 *    host before anything is enqueued.  Errors raised by the kernels (a bounded
 *    wait that gave up, an over-long decode sequence) are reported by
 *    pivot_sync_status().
 *  - There is no CPU fallback: on a machine without an sm_100 device every
 *    call returns PIVOT_ERR_UNSUPPORTED.
 */
#ifndef PIVOT_H_
#define PIVOT_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { PIVOT_REFINE = 0, PIVOT_REUSE = 1 } pivot_mode_t;

/*
 * Option bit OR-ed into `mode`: scan with the group mean rounded to bf16
 * instead of the fp32 mean.  This is a variant of the method, not the method:
 * the pages define the proxy as the group mean ("How It Works": proxy_q =
 * mean(group)) and this library takes it in fp32 by default, which the
 * tensor-core scan carries as three bf16 terms (three MMA passes per key
 * tile).  With the flag the scan makes one pass; candidate sets then differ
 * from the fp32-mean ones wherever the bf16 rounding reorders near-boundary
 * keys.
 */
enum { PIVOT_PROXY_BF16 = 0x100 };

/*
 * Option bit OR-ed into PIVOT_REFINE (prefill entry points only): the
 * listing's reading of Refine ("Show Me The Code", pivot_refine, which scans
 * k[:pos] for each member): member pos takes its candidate set from the group
 * proxy's scores over its own prefix j < pos, instead of one set per group
 * over j < last.  A fidelity variant, not the method's one shared scan: the
 * scan runs once per member (rows = positions) and every member gathers its
 * own candidates.  Its candidate rows hold L*H*ceil(Kc/128)*128 int32 of the
 * workspace; out_cand (when given) is then [L,H,Kc].  Decode entry points and
 * PIVOT_REUSE return PIVOT_ERR_INVALID_ARG with this bit.
 */
enum { PIVOT_PER_MEMBER_SCAN = 0x200 };

typedef enum {
  PIVOT_OK = 0,
  PIVOT_ERR_INVALID_ARG = 1,
  PIVOT_ERR_UNSUPPORTED = 2,
  PIVOT_ERR_CUDA = 3,
  PIVOT_ERR_TIMEOUT = 4,
  PIVOT_ERR_WORKSPACE = 5
} pivot_status_t;

/*
 * PIVOT prefill indexer for one layer, all heads.
 * Paper abstract and "How It Works": consecutive queries form groups of g
 * (starting at 0, g, 2g, ...; the last may be partial); each group's proxy is
 * the mean of its queries (fp64 sum divided by the member count, rounded to
 * fp32); one scan of the proxy over the group's causal prefix gives a
 * candidate set.
 *   mode = PIVOT_REFINE ("How It Works" per-query refine; listing pivot_refine):
 *     scan keys j < last (the group's largest position), C = top-min(Kc,last);
 *     member pos re-scores {j in C : j < pos} with its own query and keeps
 *     top-min(top_k, that count).
 *   mode = PIVOT_REUSE (listing pivot_reuse): scan keys j < s (group start);
 *     every member gets the proxy's top-min(top_k, s).  Kc is not used.
 *   Either may be OR-ed with PIVOT_PROXY_BF16 (the bf16-proxy variant);
 *   PIVOT_REFINE also with PIVOT_PER_MEMBER_SCAN (the listing's per-member
 *   scan).
 * q, k:     bf16 [L][H][d].
 * out_idx:  int32 [L][H][top_k].
 * Temporary device memory is taken with cudaMallocAsync on `stream` and freed
 * on it before return (see pivot_index_ws to supply it instead).
 */
int pivot_index(const void* q, const void* k, int L, int H, int d, int g, int top_k, int Kc, int mode,
                int32_t* out_idx, void* stream);

/*
 * Dense indexer -- the per-query scan that PIVOT replaces ("The Problem": every
 * query scores every preceding token and keeps the top-k).
 * out_idx[pos][h] = top-min(top_k, pos) of q[pos,h] . k[j,h] over j < pos.
 * q, k bf16 [L][H][d]; out_idx int32 [L][H][top_k].
 */
int dense_index(const void* q, const void* k, int L, int H, int d, int top_k, int32_t* out_idx,
                void* stream);

/*
 * PIVOT decode indexer for one multi-token-prediction step over a batch of
 * sequences (paper abstract: in decode a group is the queries decoded together
 * in one MTP step).  Sequence b holds n_b context keys plus the g keys of this
 * step in the packed cache rows cu_seqlens[b] .. cu_seqlens[b+1]-1
 * (n_b = cu_seqlens[b+1] - cu_seqlens[b] - g >= 0); its g queries sit at
 * positions n_b .. n_b+g-1.  Refine scans j < n_b+g-1 and keeps top-min(Kc, .)
 * candidates; Reuse scans j < n_b.  Indices are positions within the sequence.
 * q:          bf16 [B][g][H][d].
 * kcache:     bf16 [cu_seqlens[B]][H][d].
 * cu_seqlens: int32 [B+1], device memory, non-decreasing.
 * max_seqlen: an upper bound on cu_seqlens[b+1]-cu_seqlens[b] for every b; a
 *             longer sequence is skipped on the device and reported by
 *             pivot_sync_status() as PIVOT_ERR_INVALID_ARG.
 * out_idx:    int32 [B][g][H][top_k].
 */
int pivot_decode_index(const void* q, const void* kcache, const int32_t* cu_seqlens, int B, int H, int d,
                       int g, int top_k, int Kc, int mode, int max_seqlen, int32_t* out_idx, void* stream);

/*
 * Workspace-taking variants: identical results; `workspace` (device, 256-byte
 * aligned, owned by the caller, contents ignored) must hold at least the
 * number of bytes reported by the matching *_workspace_size call, otherwise
 * PIVOT_ERR_WORKSPACE is returned and nothing runs.  out_scores (nullable,
 * float32, same shape as out_idx) receives the score that decided each output
 * index -- the member query's score for Refine and dense, the proxy's score
 * for Reuse -- and NaN in the padding.
 */
size_t pivot_workspace_size(int L, int H, int d, int g, int top_k, int Kc, int mode);
int pivot_index_ws(const void* q, const void* k, int L, int H, int d, int g, int top_k, int Kc, int mode,
                   int32_t* out_idx, float* out_scores, void* workspace, size_t workspace_bytes, void* stream);

size_t dense_workspace_size(int L, int H, int d, int top_k);
int dense_index_ws(const void* q, const void* k, int L, int H, int d, int top_k, int32_t* out_idx,
                   float* out_scores, void* workspace, size_t workspace_bytes, void* stream);

size_t pivot_decode_workspace_size(int B, int H, int d, int g, int top_k, int Kc, int mode, int max_seqlen);
int pivot_decode_index_ws(const void* q, const void* kcache, const int32_t* cu_seqlens, int B, int H, int d,
                          int g, int top_k, int Kc, int mode, int max_seqlen, int32_t* out_idx,
                          float* out_scores, void* workspace, size_t workspace_bytes, void* stream);

/*
 * The sparse attention that consumes the index rows ("Show Me The Code": the
 * demo after pivot_refine): for query row r, head h and the valid entries J of
 * idx[r][h] (>= 0; -1 is padding),
 *     out[r][h] = sum_{j in J} softmax_j((q[r][h] . k_j) * d^-1/2) v_j,
 * with fp32 arithmetic; a row without a valid index gets zeros.
 *   q:   bf16 [R][H][d]; prefill R = L, decode R = B*g (q of pivot_decode_index).
 *   k,v: bf16; prefill [L][H][d] (index j = key row j); decode the packed cache
 *        [rows][H][d] with cu_seqlens (device [B+1], index j of sequence
 *        r / g = cache row cu_seqlens[r / g] + j); cu_seqlens NULL = prefill.
 *   idx: int32 [R][H][top_k] (the indexer's output rows); every valid index
 *        must address a key of its sequence -- it is not checked.
 *   out: float32 [R][H][d].
 * Asynchronous on `stream`; no workspace.  Returns PIVOT_OK,
 * PIVOT_ERR_INVALID_ARG or PIVOT_ERR_UNSUPPORTED (d not 64/128, no sm_100).
 */
int pivot_sparse_attention(const void* q, const void* k, const void* v, const int32_t* idx,
                           const int32_t* cu_seqlens, int R, int H, int d, int g, int top_k, float* out,
                           void* stream);

/*
 * MTP decode over a paged key cache (the layout of paged-attention serving
 * engines).  kpages: bf16 [num_pages][page_size][H][d].  block_table: int32
 * [B][max_pages] (device) maps sequence b's logical page p -- its keys
 * p*page_size .. p*page_size + page_size - 1 -- to a page of kpages.
 * seqlens: int32 [B] (device), the cache rows n_b + g that sequence b holds.
 * page_size must be a power of two and max_pages * page_size >= max_seqlen
 * (else PIVOT_ERR_INVALID_ARG).  Every page id that a sequence's first
 * seqlens[b] keys use must index a page of kpages: the tables live on the
 * device and are not checked.  Everything else -- q, the outputs, the
 * workspace (pivot_decode_workspace_size), sequences longer than max_seqlen
 * -- is as in pivot_decode_index_ws, and the results equal those of the same
 * sequences packed contiguously.
 */
int pivot_decode_index_paged(const void* q, const void* kpages, const int32_t* block_table, const int32_t* seqlens,
                             int B, int H, int d, int g, int page_size, int max_pages, int top_k, int Kc, int mode,
                             int max_seqlen, int32_t* out_idx, float* out_scores, void* workspace,
                             size_t workspace_bytes, void* stream);

/*
 * ------------------------------------------------------------------------
 * The serving step around the indexer, over a paged cache.
 *
 * A layer that keeps its keys in pages (pivot_decode_index_paged) norms and
 * rotates its queries and keys, writes the new keys and values into the pages,
 * and attends: densely over the cache, or over the index rows.  The calls below
 * share these conventions:
 *  - New tokens are numbered 0 .. T-1, sequence after sequence.  With cu (device
 *    int32 [B+1], non-decreasing) sequence b has tokens cu[b] .. cu[b+1]-1;
 *    without it every sequence has g (T = B * g).  Tokens behind cu[B] belong to
 *    no sequence: their output rows are left as they were.
 *  - seqlens[b] (device int32 [B]) is the rows that sequence b holds with its
 *    n_b new ones: new token i sits at row (position) seqlens[b] - n_b + i.
 *  - kpages, vpages: bf16 [num_pages][page_size][heads][d], page_size a power of
 *    two, fewer than 2^31 rows; block_table: int32 [B][max_pages] (device).
 *  - The device arrays are checked where they are used: a sequence whose lengths
 *    contradict each other or exceed max_pages * page_size (or max_seqlen, where
 *    given) is skipped; a row whose page is not in [0, num_pages) is not written,
 *    and read as zeros; both are reported by pivot_sync_status() as
 *    PIVOT_ERR_INVALID_ARG.
 *  - d is 64 or 128.  fp32 arithmetic; each result is rounded once.  (One more
 *    rounding in pivot_paged_attention: told there.)
 */

/* Type of a call's inputs, and how a rotation pairs the first rot_dim channels:
 * (i, i + rot_dim/2), or (2i, 2i+1). */
typedef enum { PIVOT_BF16 = 0, PIVOT_FP16 = 1, PIVOT_FP32 = 2 } pivot_dtype_t;
#define PIVOT_CLEAR_LEFT_OUT 0x100 /* option bit of pivot_paged_append's dtype */
typedef enum { PIVOT_ROPE_HALF = 0, PIVOT_ROPE_INTERLEAVED = 1 } pivot_rope_layout_t;

/* Head rows [T][heads][d] of new tokens, strides in elements (each row must
 * start on a 16-byte boundary; channels are adjacent), with the weight [d] of
 * the norm of each head, in the same type (NULL: no norm). */
typedef struct {
  const void* data;
  const void* weight;
  long long token_stride;
  long long head_stride;
  int heads;
} pivot_heads_t;

/* The rotation, and the norm's eps.  freqs: fp64 [rot_dim/2] (device), radians a
 * position of each pair, whatever scaling made them; NULL: no rotation.
 * amplitude multiplies the cosines and sines (1 without scaling).  rot_dim is a
 * multiple of 16, at most d; channels behind it are passed on. */
typedef struct {
  const double* freqs;
  double amplitude;
  double eps;
  int rot_dim;
  int layout;
} pivot_rope_t;

/*
 * Norm and rotation of query and key heads in one pass: for each head row x of a
 * token at position pos, x_c <- x_c (mean x^2 + eps)^-1/2 w_c where a weight is
 * given, then each pair (a, b) of the first rot_dim channels becomes
 * amplitude * (a cos t - b sin t, b cos t + a sin t), t = pos * freqs[i].
 * positions: int32 [T] (device).  q or k may be NULL.  The angle is reduced in
 * fp64, so any int32 position is exact to fp32.
 * out_q, out_k: bf16 [T][heads][d], contiguous; they may be the inputs
 * themselves (bf16, contiguous), and must not overlap them otherwise.
 */
int pivot_qk_rope(const pivot_heads_t* q, const pivot_heads_t* k, int dtype, const int32_t* positions,
                  const pivot_rope_t* rope, int T, int d, void* out_q, void* out_k, void* stream);

/*
 * Writes the new keys (normed and rotated as above, at their rows' positions)
 * and values (NULL: a cache of keys alone) into their pages, and, where q is
 * given, norms and rotates the tokens' queries into out_q (bf16 [T][heads][d],
 * contiguous; it may be q itself, as above) in the same launch.  The new tokens'
 * rows must be in pages of their own: two sequences that write the same row race.
 * A token of a skipped sequence, and one whose page is not in the cache, is left
 * out: neither its row nor its queries are written.  With PIVOT_CLEAR_LEFT_OUT
 * in dtype the queries of such tokens, and of those behind cu_new[B], become zeros
 * (for an out_q that holds nothing yet).
 */
int pivot_paged_append(const pivot_heads_t* k, const pivot_heads_t* v, const pivot_heads_t* q, int dtype,
                       const pivot_rope_t* rope, const int32_t* block_table, const int32_t* seqlens,
                       const int32_t* cu_new, int T, int B, int d, int g, int num_pages, int page_size, int max_pages,
                       void* kpages, void* vpages, void* out_q, void* stream);

/* scale: of the scores (> 0).  include_self: a query at position pos sees the
 * keys j <= pos; 0: j < pos, the keys that the indexer selects from. */
typedef struct {
  double scale;
  int include_self;
} pivot_attend_t;

/*
 * Dense causal attention of the new tokens over the paged cache (their own keys
 * and values already appended): for query head h and the keys of head
 * h / (Hq / Hk),
 *     out = sum_j softmax_j(scale q . k_j) v_j,  lse = log sum_j exp(scale q . k_j)
 * over the keys that the query sees; a query that sees none, and every query of
 * a skipped sequence, gets zeros and lse = -inf.
 * q, out: bf16 [T][Hq][d], apart from one another; out_lse: float32 [T][Hq] or
 * NULL.  options NULL:
 * scale d^-1/2, include_self.  max_seqlen: an upper bound on seqlens[b]; a
 * longer sequence is skipped.  With cu_q, g is an upper bound on a sequence's new
 * tokens, for the choice of kernels alone, or 0.  Keys and values that a query
 * does not see may hold anything; of those that it sees, an infinite or NaN value
 * makes its channel so, however small its weight.  workspace as in the _ws
 * variants; the size may be 0.
 * Scores, the softmax's sums and the results' are fp32.  Each weight is rounded to
 * bf16 for its product with the values (the matrix instructions' operand type), and
 * out to bf16: an error of at most 2^-8 (sum_j p_j |v_j| + |out|) beside fp32's, p
 * being the softmax; as the weights' roundings differ, in truth about
 * 2^-8 (sqrt(sum_j p_j^2 v_j^2) + |out|).  out_lse has none of it.
 */
size_t pivot_paged_attention_workspace_size(int T, int B, int Hq, int Hk, int d, int max_seqlen);
int pivot_paged_attention(const void* q, const void* kpages, const void* vpages, const int32_t* block_table,
                          const int32_t* seqlens, const int32_t* cu_q, const pivot_attend_t* options, int T, int B,
                          int Hq, int Hk, int d, int g, int num_pages, int page_size, int max_pages, int max_seqlen,
                          void* out, float* out_lse, void* workspace, size_t workspace_bytes, void* stream);

/*
 * pivot_sparse_attention over a paged cache: q bf16 [B][g][H][d], idx int32
 * [B][g][H][top_k] (the rows of pivot_decode_index_paged; top_k at most 2^30), out
 * float32 [B][g][H][d].  An index at or beyond seqlens[b], or whose page is not in the
 * cache, is left out and reported; a skipped sequence's rows are zeros.
 */
int pivot_sparse_attention_paged(const void* q, const void* kpages, const void* vpages, const int32_t* block_table,
                                 const int32_t* seqlens, const int32_t* idx, int B, int H, int d, int g, int num_pages,
                                 int page_size, int max_pages, int top_k, float* out, void* stream);

/*
 * As the _ws variants, with two more nullable outputs that expose the
 * method's intermediate results ("How It Works": the proxy of each group and
 * its candidate set C = top-Kc of the proxy scores):
 *   out_proxy: float32 [G][H][d] (decode: [B][H][d]), each group's proxy --
 *              the fp32 mean of its queries (or its bf16 rounding under
 *              PIVOT_PROXY_BF16), 16-byte aligned;
 *   out_cand:  int32 [G][H][Kc] (decode: [B][H][Kc]), PIVOT_REFINE only (else
 *              PIVOT_ERR_INVALID_ARG): each group's candidate key indices in
 *              ascending order, -1 padded; a decode sequence skipped for its
 *              length gets an all -1 row.
 * G = ceil(L / g).
 */
int pivot_index_ex(const void* q, const void* k, int L, int H, int d, int g, int top_k, int Kc, int mode,
                   int32_t* out_idx, float* out_scores, float* out_proxy, int32_t* out_cand, void* workspace,
                   size_t workspace_bytes, void* stream);
int pivot_decode_index_ex(const void* q, const void* kcache, const int32_t* cu_seqlens, int B, int H, int d, int g,
                          int top_k, int Kc, int mode, int max_seqlen, int32_t* out_idx, float* out_scores,
                          float* out_proxy, int32_t* out_cand, void* workspace, size_t workspace_bytes,
                          void* stream);

/*
 * Decode without any device allocation (the paper has no counterpart; this is
 * a deployment variant of pivot_decode_index, same arguments and results).
 * For callers that cannot allocate device memory during a decode step: an
 * inference engine that has already handed all free HBM to its KV-cache pool,
 * so a cudaMalloc there would fail or fragment it, or host code that has no
 * allocator of its own and must not own device buffers.  Its scratch is a
 * 32 MiB array built into the library (held by every GPU that loads it until
 * the process exits); a call whose scratch need -- proxies B*H*d*4 + order keys
 * H*B*max_seqlen*4 + (Refine) candidates H*B*CW*4 bytes, CW = Kc rounded up to
 * a multiple of 128, each rounded up to 256 -- exceeds 32 MiB is rejected with
 * PIVOT_ERR_WORKSPACE and a message.
 * The first call on each device looks the array's address up (once, with that
 * device current); make that first call before any stream capture.  All calls
 * share the one array and it keeps the previous call's contents (nothing in it
 * needs to start at zero): calls that may overlap on the GPU -- concurrent
 * streams, or several host threads -- race on it and must be serialised by the
 * caller.
 */
int pivot_decode_index_noalloc(const void* q, const void* kcache, const int32_t* cu_seqlens, int B, int H, int d,
                               int g, int top_k, int Kc, int mode, int max_seqlen, int32_t* out_idx,
                               float* out_scores, void* stream);

/*
 * Synchronises `stream`, then reads and clears this device's kernel status
 * word.  Returns PIVOT_OK, PIVOT_ERR_TIMEOUT (a bounded wait inside a kernel
 * gave up; that call's outputs are not valid), PIVOT_ERR_INVALID_ARG (status bit
 * 2: a sequence exceeded max_seqlen or its block table, held fewer rows than its
 * new tokens, or had offsets that do not fit; or bit 16: a page outside the cache
 * or an index outside its sequence) or PIVOT_ERR_CUDA (a CUDA error, or status bit
 * 8: a refine selection exceeded its round limit, which finite scores never
 * do; that call's outputs are not valid).  *flags (nullable) receives the raw
 * status bits; bit 4 means some rows took the exact fallback path (results
 * remain exact).
 */
int pivot_sync_status(void* stream, int* flags);

/*
 * Launch trace (profiling aid, off by default; per calling thread).  While
 * enabled, every kernel launch of this library is bracketed by two CUDA events
 * recorded on the launch stream.  pivot_trace_collect() waits for the recorded
 * events, aggregates them by kernel name and clears the trace: names receives a
 * comma-separated list, ms[i] the summed device time of kernel i, count[i] its
 * launches (up to max_items kernels).  Returns the number of kernels, or a
 * negated error code.
 */
int pivot_trace_enable(int on);
int pivot_trace_collect(char* names, size_t names_len, float* ms, int* count, int max_items);

/*
 * Testing aid (the method has no counterpart).  Every wait of a kernel on
 * another of its roles (an mbarrier phase) gives up after a limit, raises the
 * status that pivot_sync_status() reports as PIVOT_ERR_TIMEOUT, drains what it
 * had issued and returns; no kernel traps or spins for ever.  This sets that
 * limit, in nanoseconds, for the calls that follow in this process (0 restores
 * the default of 2 seconds).  A tiny limit makes a call time out on purpose;
 * its outputs are then not valid.  Returns PIVOT_OK.
 */
int pivot_set_wait_limit(unsigned long long ns);

/* Message of the last error on the calling thread ("" if none). */
const char* pivot_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* PIVOT_H_ */
