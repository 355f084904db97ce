/*
 * ltk.h -- C ABI of the GB300 fused Indexer-TopK library (libltk.so).
 *
 * The operation (LiteTopK: "Exploiting the Curse of Dimensionality for a Fused
 * Indexer-TopK Kernel in Long-Context Sparse Attention", gist.science technical
 * summary, Problem Statement and Methodology):
 *
 *   for each query t of a prefill chunk and every key s visible to it
 *   (causal: s <= positions[t]) compute the indexer score
 *
 *       I[t,s] = sum_h w[t,h] * ReLU(q[t,h,:] . k[s,:])
 *
 *   (the DeepSeek Sparse Attention indexer score, named I_{t,s} in the
 *   summary's bin map) and return the exact top-k keys of each query, without
 *   writing the T x S score matrix to device memory.  The library runs the
 *   summary's three stages -- Sample (Methodology step 1), Filter (step 2) and
 *   Select (step 3) -- as CUDA kernels for sm_103a.
 *
 * Conventions shared by every entry point
 *   - Pointers named "device" must point to device memory of the current
 *     device; they stay owned by the caller.  Every device pointer must be
 *     16-byte aligned (TMA requirement); misaligned pointers fail with
 *     LTK_ERR_ARG.
 *   - "stream" is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  Compute calls are asynchronous on that stream and never
 *     synchronise the host, except where stated.
 *   - Arguments are validated on the host before any launch; a bad argument
 *     returns LTK_ERR_ARG and enqueues nothing.
 *   - Output order: each query's k slots hold the selected keys sorted by
 *     (score descending, key index ascending); slots beyond min(k, V_t), V_t
 *     the number of visible keys, hold index -1 and score -inf.
 *   - Errors raised on the device (a bounded wait that timed out) are
 *     recorded in a status word that ltk_get_stats reports.
 *   - A handle is not thread-safe: calls on one handle must be serialised,
 *     and two calls on one handle must not overlap on the GPU (they share the
 *     handle's workspace), i.e. issue them on one stream or synchronise.
 */
#ifndef LTK_H
#define LTK_H

#ifdef __cplusplus
extern "C" {
#endif

#define LTK_ABI_VERSION 2

typedef enum {
  LTK_OK = 0,
  LTK_ERR_ARG = 1,          /* invalid argument; nothing was enqueued         */
  LTK_ERR_CUDA = 2,         /* a CUDA runtime/driver call failed              */
  LTK_ERR_NOMEM = 3,        /* workspace allocation failed                    */
  LTK_ERR_OVERFLOW = 4,     /* informational: candidate list overflowed; the
                               affected queries were recomputed exactly      */
  LTK_ERR_TIMEOUT = 5,      /* a bounded device-side wait expired             */
  LTK_ERR_UNSUPPORTED = 6   /* shape or mode the library does not implement   */
} ltk_status;

/* LTK_F16 is a type of the paged cache's inputs and of logits only, LTK_F32 of logits. */
typedef enum { LTK_BF16 = 0, LTK_FP8_E4M3 = 1, LTK_F16 = 2, LTK_F32 = 3 } ltk_dtype;

/*
 * Handle configuration (fixed at ltk_create).
 *   heads, dim      H and d of q[T,H,d] and k[S,d] (see engine for the shapes
 *                   each kernel serves).
 *   dtype           LTK_BF16, or LTK_FP8_E4M3 with per-token fp32 scales
 *                   (q_scale[T], k_scale[S]; the value is code * scale).
 *   relu, causal    1 for the indexer score (ReLU per head, key s visible iff
 *                   s <= positions[t]).
 *   max_T, max_S    largest chunk and key cache the workspace is sized for.
 *   k               largest k a call may request (<= 8192).
 *   n_bins          equal-width bins of the Filter stage's gate
 *                   (Methodology step 2, "Bin Mapping"); power of two in
 *                   [32, 512] for bf16, [32, 2048] for fp8.
 *   cand_cap        per-query capacity of the candidate list written by the
 *                   Filter stage; 0 derives it from k and max_S.
 *   sample_size     k' = number of sample keys (Methodology step 1 uses
 *                   k' = 3k); 0 means 3k.  At most 16384.
 *   seed            seed of the random sample used when no previous-chunk
 *                   sample is given.
 *   refresh_interval  key tiles (128 keys) between threshold refreshes by the
 *                   refresh warp ("Threshold Refresh"); 0 disables refresh.
 *   enable_decoupled  1 also allocates the max_T x max_S fp32 score matrix of
 *                   the decoupled baseline (ltk_decoupled_topk).
 *   rescue_rows     queries recomputed concurrently when a candidate list
 *                   overflows (each holds a max_S fp32 score row); 0 = 16.
 *   enable_host_io  1 also allocates device staging for ltk_indexer_topk_host.
 *   engine          0 (auto): the tensor-core kernels where the shape allows
 *                   (H = 64 and d = 128 with ReLU; or H = 1, bf16, no mask),
 *                   otherwise the CUDA-core kernel; 1: tensor cores only;
 *                   2: the CUDA-core kernel with the fused affine bin map
 *                   (any 1 <= H <= 128, d a multiple of 8 -- of 16 for
 *                   e4m3 -- up to 4096, H * d * 4 + n_bins * 4 <= 100 KB).
 *   debug_flags     0 in normal use.  Bit 0 (tests of failure handling): the
 *                   Filter kernel's producer issues no key-tile loads, so its
 *                   bounded waits expire (about 2 s), the kernel records
 *                   LTK_ERR_TIMEOUT, releases its resources and returns; the
 *                   outputs are then undefined and ltk_get_stats reports the
 *                   status.
 */
typedef struct {
  int heads;
  int dim;
  int dtype;
  int relu;
  int causal;
  int max_T;
  long long max_S;
  int k;
  int n_bins;
  int cand_cap;
  int sample_size;
  unsigned long long seed;
  int refresh_interval;
  int enable_decoupled;
  int rescue_rows;
  int enable_host_io;
  int engine;
  int debug_flags;
} ltk_config;

typedef struct ltk_handle ltk_handle;

/*
 * Per-call statistics of the last compute call on a handle.  Reading them
 * synchronises the stream of that call.
 *   cand_written   candidates that passed the gate, summed over queries
 *                  (bytes written per query = 8 * cand_written / T + 8 * k).
 *   cand_max       largest per-query candidate count.
 *   n_overflow     queries whose list exceeded cand_cap (recomputed exactly).
 *   device_status  first error code raised on the device, 0 if none.
 *   visible_pairs  query-key pairs the last call scored (sum of V_t).
 *   ms_*           stage times from CUDA events recorded on each call's
 *                  stream while timing is enabled (ltk_set_timing), averaged
 *                  over the last timed_calls calls (at most 64) since timing
 *                  was last enabled; -1 when no call was timed.
 *   launches       kernels this library launched in the process so far.
 */
typedef struct {
  int T;
  long long S;
  int k;
  long long visible_pairs;
  long long cand_written;
  int cand_max;
  int n_overflow;
  int device_status;
  float ms_sample;
  float ms_filter;
  float ms_select;
  float ms_rescue;
  float ms_total;
  int timed_calls;
  long long launches;
} ltk_stats;

/* ABI version of the loaded library (LTK_ABI_VERSION). */
int ltk_abi_version(void);

/* Static text of a status code. */
const char* ltk_status_string(int status);

/* Fills *cfg with defaults for the indexer (bf16, ReLU, causal, n_bins 512,
 * refresh every tile, derived cand_cap, k' = 3k).  Host only. */
ltk_status ltk_config_init(ltk_config* cfg, int heads, int dim, int k, int max_T,
                           long long max_S);

/* Device bytes ltk_create would allocate for *cfg.  Host only (no CUDA
 * call); LTK_ERR_ARG / LTK_ERR_UNSUPPORTED for an invalid configuration. */
ltk_status ltk_workspace_bytes(const ltk_config* cfg, unsigned long long* bytes);

/* Validates *cfg and allocates the handle and its device workspace on the
 * current device.  The workspace is owned by the handle. */
ltk_status ltk_create(const ltk_config* cfg, ltk_handle** out);

/* Frees the handle and its workspace (synchronises the device first).
 * NULL is accepted. */
void ltk_destroy(ltk_handle* h);

/* Enables (1) or disables (0) per-stage CUDA-event timing on later calls;
 * enabling also restarts the averaging window of ltk_get_stats. */
ltk_status ltk_set_timing(ltk_handle* h, int enable);

/*
 * Seeded random sample for a first chunk (Methodology step 1 contrasts the
 * previous-chunk sample with random sampling): n distinct key ids drawn one
 * per stratum of [0, S), written to sample_out[n] (device int32).
 */
ltk_status ltk_random_sample(ltk_handle* h, long long S, int n, int* sample_out,
                             void* stream);

/*
 * Previous-chunk sample (Methodology step 1: reuse the top-k' tokens of the
 * previous chunk's results, k' = 3k).  prev_idx[T_prev, k_prev] (device int32)
 * is the previous chunk's output; entries < 0 or >= S are ignored.  Key ids
 * are ranked by how many of the previous chunk's queries selected them (ties:
 * higher id first); if fewer than n ids were selected at all, the rest is
 * filled with pseudo-random unselected ids.  Writes n distinct ids to
 * sample_out[n] (device).  Requires n <= S and S <= max_S.
 */
ltk_status ltk_make_sample(ltk_handle* h, const int* prev_idx, int T_prev, int k_prev,
                           long long S, int n, int* sample_out, void* stream);

/*
 * Fused Indexer-TopK (Sample -> Filter -> Select).
 *   q          device [T, H, d] bf16 or e4m3, row-major.
 *   q_scale    device [T] fp32 (e4m3 only, > 0), else NULL.
 *   w          device [T, H] fp32 head weights (any sign).
 *   k_cache    device [S, d] bf16 or e4m3, row-major.
 *   k_scale    device [S] fp32 (e4m3 only, > 0), else NULL.
 *   positions  device [T] int32 absolute query positions (causal mask);
 *              ignored when the handle is not causal.
 *   prev_topk  device int32 sample key ids (e.g. from ltk_make_sample), or
 *              NULL for a seeded random sample of sample_size keys.  Ids
 *              outside [0, S) and duplicates are dropped; ids invisible to a
 *              query are skipped for that query.  n_prev <= 16384.
 *   k          1 <= k <= cfg.k.
 *   out_idx    device [T, k] int32; out_score device [T, k] fp32 (the
 *              kernel's fp32 score of each selected key).
 * 0 <= T <= max_T, 1 <= S <= max_S.  T == 0 enqueues nothing.
 * The call neither synchronises nor allocates, so it can be captured in a CUDA
 * graph (stream capture) and replayed: the graph reads the buffers named here
 * at replay time, and a replay overwrites the handle's statistics like a call.
 * Make one call on the handle outside capture first (it sets kernel
 * attributes on the device), and keep timing off while capturing.
 */
ltk_status ltk_indexer_topk(ltk_handle* h, const void* q, const float* q_scale,
                            const float* w, const void* k_cache, const float* k_scale,
                            const int* positions, int T, long long S,
                            const int* prev_topk, int n_prev, int k,
                            int* out_idx, float* out_score, void* stream);

/*
 * Same contract as ltk_indexer_topk, but every pointer is HOST memory
 * (pinned for asynchronous copies).  The library copies the inputs into its
 * own device staging (enable_host_io), runs the fused path and copies the
 * results back; the call returns once the results are in out_idx/out_score.
 */
ltk_status ltk_indexer_topk_host(ltk_handle* h, const void* q, const float* q_scale,
                                 const float* w, const void* k_cache, const float* k_scale,
                                 const int* positions, int T, long long S,
                                 const int* prev_topk, int n_prev, int k,
                                 int* out_idx, float* out_score, void* stream);

/*
 * Decoupled baseline (the DSA-style two-stage design the summary's Problem
 * Statement describes): write the full fp32 score matrix [T, S] to device
 * memory with the same tensor-core scorer, then run a radix select over each
 * row, reading it several times.  Same arguments and output contract as
 * ltk_indexer_topk (no sample).  Needs enable_decoupled.
 */
ltk_status ltk_decoupled_topk(ltk_handle* h, const void* q, const float* q_scale,
                              const float* w, const void* k_cache, const float* k_scale,
                              const int* positions, int T, long long S, int k,
                              int* out_idx, float* out_score, void* stream);

/*
 * Decoupled top-k that allocates nothing (no counterpart in the paper: it is
 * an integration convenience).  For callers that cannot call cudaMalloc -- a
 * plugin inside an engine that owns all device memory through its own pool,
 * or a latency-critical path where cudaMalloc's implicit device
 * synchronisation is not acceptable.  Same computation and output contract as
 * ltk_decoupled_topk for H = 64, d = 128, ReLU scores, without a handle:
 * dtype is LTK_BF16 or LTK_FP8_E4M3, causal selects the s <= positions[t]
 * mask.  Its scratch, the T x S fp32 score matrix, lives in a static device
 * array of 4,194,304 floats (16 MiB) that every GPU loading the library
 * holds until process exit; T * S above that returns LTK_ERR_ARG.  The
 * caller still owns all inputs and outputs.
 *   device_status  device int (4-byte aligned, caller-owned) or NULL.  The
 *                  call zeroes it on the stream; a bounded wait in the scorer
 *                  that expires (about 2 s) stores LTK_ERR_TIMEOUT there, and
 *                  the outputs of that call are then undefined.  Read it after
 *                  the stream has finished the call.  With NULL such an error
 *                  is not reported anywhere.
 * Each call looks up the array's device address with the caller's device
 * current (no allocation); the first call on a device also loads the
 * library's kernels there and sets their attributes, so make it before any
 * stream capture.  All calls share the array, so calls that overlap on the
 * GPU race and corrupt each other's results: serialise them (one stream, or
 * synchronise between calls).
 */
ltk_status ltk_decoupled_topk_noalloc(int dtype, int causal, const void* q, const float* q_scale,
                                      const float* w, const void* k_cache, const float* k_scale,
                                      const int* positions, int T, long long S, int k,
                                      int* out_idx, float* out_score, int* device_status,
                                      void* stream);

/*
 * LiteDSA candidate packing (LiteTopK arXiv abstract: LiteDSA packs the
 * overlapping candidates of neighbouring query tokens into a shared key/value
 * list for joint attention, with per-query masks that keep each token's own
 * top-k membership).  Consecutive queries form groups of `group`; for group g
 * (queries g*group .. g*group+group-1, the last group may be short):
 *   union_idx  device int32 [ceil(T/group), group*k]: the ascending set union
 *              of the group's valid (>= 0) indices, padded with -1;
 *   union_len  device int32 [ceil(T/group)]: number of valid union entries;
 *   masks      device uint32 [T, ceil(group*k/32)]: bit j of query t's row is
 *              set iff union entry j of t's group is one of t's indices.
 * topk_idx is device int32 [T, k] (e.g. ltk_indexer_topk's out_idx; a row
 * holds distinct indices, -1 = empty slot).  No handle, no allocation.
 * group in [1, 256]; group*k <= 16384 and the group's shared-memory footprint
 * (sorted keys + masks) <= 200 KB, else LTK_ERR_UNSUPPORTED.
 */
ltk_status ltk_litedsa_pack(const int* topk_idx, int T, int k, int group, int* union_idx,
                            int* union_len, unsigned int* masks, void* stream);

/*
 * Paged key/value cache held in 8 bits, and the attention that reads it (the
 * layer around the indexer: keys and values are appended, the indexer chooses
 * keys, the attention reads them).
 *
 * Cache of one layer (device memory, owned by the caller):
 *   k_codes, v_codes  e4m3 codes [num_pages, heads, page, dim];
 *   k_scale, v_scale  fp32 [num_pages, heads], 0 or 2^-64 to 2^64; the value held
 *                     is code * scale (a scale of 0: zeros).
 * page is 16, 32, 64 or 128 tokens, dim 64 or 128.
 *
 * A handle binds the four buffers and owns a workspace of a few tens of MiB on
 * the device it was created on.  Calls on one handle must not overlap on the
 * GPU (one stream, or synchronise).  They neither allocate nor synchronise and
 * read the batch on the device, so they can be captured in a CUDA graph.
 */
typedef struct {
  long long num_pages;
  int heads;
  int dim;
  int page;
  int engine;        /* attention kernel: 0 chosen by measured costs (see kv_api.cu),
                        1 the one for few rows per KV head, 2 the tensor-core tiles */
  void* k_codes;
  void* v_codes;
  float* k_scale;
  float* v_scale;
} ltk_kv_config;

typedef struct ltk_kv ltk_kv;

/*
 * The step's batch: B sequences with N new tokens (queries) in all.
 *   page_table  device int32 [B, table_width]: pages of each sequence in order;
 *   seq_lens    device int32 [B]: cached tokens of each sequence, this step's
 *               new ones among them;
 *   cu_q        device int32 [B + 1]: tokens cu_q[b] .. cu_q[b+1]-1 are
 *               sequence b's (0 of them is allowed), cu_q[B] = N.
 * New token i of sequence b has position seq_lens[b] - n_b + i, n_b its number
 * of new tokens.  Its position p is row p % page of page page_table[b, p / page].
 * table_width * page is below 2^31; positions from 2^31 - 1024 on count as past
 * the table.
 * Set the handle's device status to LTK_ERR_ARG: a page number outside
 * [0, num_pages) and a position past the page table's columns (append writes
 * nothing there, queries that see it get NaN); in append also a sequence shorter
 * than its new tokens (none of them is stored) and a position past the rotation
 * table (the token is held as NaN).  In attention the queries before a sequence's
 * first token see nothing (0 and -inf) and are not reported.
 * A cu_q that does not rise from 0 to N is clamped to that range: no call reads
 * or writes outside the buffers and the pages of the table for it, but what its
 * tokens get is not defined, and only the dense tensor-core kernel (engine 2;
 * never chosen for 16 rows per KV head or fewer) reports it.
 */
typedef struct {
  const int* page_table;
  int table_width;
  const int* seq_lens;
  const int* cu_q;
  int B;
  int N;
} ltk_kv_batch;

ltk_status ltk_kv_create(const ltk_kv_config* cfg, ltk_kv** out);

/* Frees the handle and its workspace (synchronises the device first), not the
 * cache.  NULL is accepted. */
void ltk_kv_destroy(ltk_kv* h);

/*
 * Appends the batch's N new tokens.
 *   dtype       LTK_BF16 or LTK_F16: type of k, v, q and q_out.
 *   k, v        device [N, heads, dim]; consecutive tokens k_stride / v_stride
 *               elements apart (a multiple of 8, so slices of a fused
 *               projection's output serve as they are).
 *   cos_table,  device fp32 [table_rows, rot / 2], row p the angles of position
 *   sin_table   p, or both NULL for no rotation.  The first rot elements of each
 *               key (and query) head are rotated, rot a multiple of 16:
 *               elements i and i + rot/2 form a pair, or 2i and 2i + 1 when
 *               interleaved is 1.
 *   q, q_out    device [N, q_heads, dim], rotated the same way from q (tokens
 *               q_stride elements apart) to the contiguous q_out; both NULL to
 *               leave queries out.  q_out must not overlap q, except that
 *               q_out == q with contiguous tokens rotates in place.
 * Each touched (page, head) gets the scale 2^e, e the smallest exponent >= -40
 * with max|x| <= 448 * 2^e over its tokens; a page that already held tokens
 * never lowers e, and when e grows its held codes are rounded again (also when a
 * scale of the caller's own is no power of two: e is then the next one above).
 * A token whose key or value row of a head holds a NaN, an infinity or a value
 * beyond 448 * 2^40 is held in that head as a NaN key row and a zero value row: every
 * query that sees it gets NaN, no other query does.
 */
ltk_status ltk_kv_append(ltk_kv* h, const ltk_kv_batch* batch, int dtype, const void* k,
                         long long k_stride, const void* v, long long v_stride,
                         const float* cos_table, const float* sin_table, int table_rows, int rot,
                         int interleaved, const void* q, long long q_stride, int q_heads,
                         void* q_out, void* stream);

/*
 * Attention of the batch's N queries over their sequences' cached tokens:
 *   out = softmax(scale * q . K) V over keys j with j <= p (p the query's
 *   position) and, when window > 0, j > p - window or j < sinks.
 *   q           device [N, q_heads, dim], tokens q_stride elements apart;
 *               q_heads a multiple of the cache's heads; query head i reads KV
 *               head i / (q_heads / heads).
 *   max_q       the largest number of queries of one sequence, as a hint for the
 *               choice of kernel (0: unknown); results are right for any value, but
 *               one far from the truth can take a slower kernel.
 *   out         device [N, q_heads, dim] in dtype;  lse device fp32 [N, q_heads]
 *               (natural logarithm of the sum of exponentials) or NULL.
 * A query that sees no key gets 0 and -inf.  Value codes must not be NaN
 * (ltk_kv_append never writes one); rows past a sequence's length are not read.
 * out must not overlap q.
 * Arithmetic: products of f16 numbers (codes exactly, queries after a scaling by
 * powers of two, weights rounded to f16); sums and softmax statistics in fp32.
 * Keys whose weight times value scale is below 2^-21 of the row's largest keep
 * fewer bits, below 2^-31 none.  For listed keys and more than 64 query heads a
 * KV head the same holds of block scales below 2^-21 of the largest among 16
 * entries of the list.  A value scale is added to the score as its logarithm, so
 * weights carry the score's rounding to fp32, which passes f16's at scores of 10^4.
 */
ltk_status ltk_kv_attention(ltk_kv* h, const ltk_kv_batch* batch, int dtype, const void* q,
                            long long q_stride, int q_heads, int max_q, float scale, int window,
                            int sinks, void* out, float* lse, void* stream);

/*
 * The same over chosen keys: idx device int32 [N, k] holds distinct positions in
 * each query's own sequence (ltk_indexer_topk's out_idx when the chunk is one
 * sequence); an entry below 0 or beyond the query's position is an empty slot.
 */
ltk_status ltk_kv_attention_selected(ltk_kv* h, const ltk_kv_batch* batch, int dtype, const void* q,
                                     long long q_stride, int q_heads, const int* idx, int k,
                                     float scale, void* out, float* lse, void* stream);

/*
 * Attention of sequences that begin with the same pages, their common part read
 * once for all of them (many continuations of one prompt, requests behind one
 * document).  Arguments and results are those of ltk_kv_attention without a
 * window; only the work is shared out differently.
 *   groups      device int32 [num_groups + 1], rising from 0 to B: sequences
 *               groups[g] .. groups[g+1]-1 are group g; NULL: all are one group.
 *   workspace   device, 16-byte aligned, workspace_bytes long, at least what
 *               ltk_kv_shared_bytes says; its contents do not outlast the call.
 * What a group shares is found on the device: the pages with which the table
 * rows of its sequences begin alike, cut to whole pages that all their queries
 * see.  A sequence without queries, without a whole page before its first query
 * or with another first page than the group's first that has one takes no part
 * (it is attended to by itself, though its queries go through the shared part's products too).  One
 * part is shared by all that take part: a sequence with one page in common leaves one page
 * for its whole group, so a group is best made of sequences that have about as much in common.  Groups that do not rise from 0 to B set the
 * device status to LTK_ERR_ARG, and nothing is shared.
 * The shared and the own part of a row are joined in fp32; each is rounded as
 * in ltk_kv_attention.
 */
ltk_status ltk_kv_attention_shared(ltk_kv* h, const ltk_kv_batch* batch, const int* groups, int num_groups,
                                   int dtype, const void* q, long long q_stride, int q_heads, int max_q,
                                   float scale, void* out, float* lse, void* workspace,
                                   unsigned long long workspace_bytes, void* stream);

/* Bytes of workspace that a call with B sequences and N queries of q_heads heads needs. */
ltk_status ltk_kv_shared_bytes(const ltk_kv* h, int B, int N, int q_heads, unsigned long long* bytes);

/*
 * Reads tokens back: of each sequence the last cu_q[b+1] - cu_q[b] of its
 * seq_lens[b] tokens, in the batch's order (the batch of an append, or one with
 * cu_q the running sum of seq_lens for whole sequences).
 *   dtype        LTK_BF16 or LTK_F16: type of k_out and v_out;
 *   cos_table ..  as in ltk_kv_append: keys are rotated back by their positions'
 *                angles; NULL: keys as they are held;
 *   k_out, v_out device [N, heads, dim], contiguous.
 * Values are code * scale in fp32 (zeros where the scale is 0), rounded once.  A
 * token whose page is outside the pool or past the table, that lies before its
 * sequence's first (more tokens asked for than there are) or past the rotation
 * table is NaN, and the device status is set to LTK_ERR_ARG.  Rows of no
 * sequence are left as they were.
 */
ltk_status ltk_kv_read(ltk_kv* h, const ltk_kv_batch* batch, int dtype, const float* cos_table,
                       const float* sin_table, int table_rows, int rot, int interleaved, void* k_out,
                       void* v_out, void* stream);

/* First error raised on the device by the handle's calls so far (0: none) and
 * clears it; synchronises the stream. */
ltk_status ltk_kv_status(ltk_kv* h, int* device_status, void* stream);

/*
 * Draws a token for each row of logits from a given random number.
 *   logits  device [B, V] of LTK_BF16, LTK_F16 or LTK_F32, rows row_stride
 *           elements apart, aligned to their elements; up to 360,000 tokens of 32
 *           bits or 720,000 of 16 (else LTK_ERR_UNSUPPORTED);
 *   s       the settings, for each row (device pointers [B]) or, where a pointer
 *           is NULL, one for all;
 *   u       device fp32 [B]: random numbers in [0, 1);
 *   token   device int32 [B];  logp  device fp32 [B]: the natural logarithm of the
 *           token's probability among those it was drawn from.
 * With w_i = exp((x_i - max x) / temperature) and tokens ordered by (x descending,
 * index ascending), the following are left, each step among those of the one before:
 *   min_p   those with w_i >= min_p (0: all);
 *   top_k   the first top_k (0 or less, or V or more: all);
 *   top_p   the fewest first ones whose weights sum to top_p of the total or
 *           more, at least one (1 or more: all).
 * The token is the first of these, in the order of indices, at which the running
 * sum of weights exceeds u times their total (u below 0 counts as 0, from 1 on as
 * the largest below 1).  Temperature 0 (and any below 2^-127) takes the largest
 * logit, the first of equal ones, with logp 0.  Logits of -inf are never drawn; a row of nothing else gives
 * -1 and -inf, a row with a NaN or +inf, or with a setting out of range
 * (temperature below 0, infinite or NaN, top_p below 0 or NaN, min_p outside
 * [0, 1], u NaN), -1 and NaN.
 * Weights are whole numbers in units of 2^-44 of (about) the largest, right to
 * 2^-30.5 of themselves and that unit (those below 2^-42 are never drawn; with temperatures
 * above 2^100, logits above 2^114 have weights of fewer bits), their sums exact: a row's
 * result depends on its logits and settings only.  Needs no handle or workspace, neither allocates nor synchronises.
 */
typedef struct {
  const float* temperature;
  const int* top_k;
  const float* top_p;
  const float* min_p;
  float temperature_all;
  int top_k_all;
  float top_p_all;
  float min_p_all;
} ltk_sampling;

ltk_status ltk_sample_tokens(const void* logits, int dtype, long long row_stride, int B, int V,
                             const ltk_sampling* s, const float* u, int* token, float* logp, void* stream);

/* Statistics of the last compute call (synchronises its stream). */
ltk_status ltk_get_stats(ltk_handle* h, ltk_stats* out);

#ifdef __cplusplus
}
#endif

#endif /* LTK_H */
