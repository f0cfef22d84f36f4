/*
 * daa.h -- C ABI of libdaa: paged KV append and mixed-batch paged attention
 * (chunked-prefill requests and decode requests in one batch) for sm_103a.
 *
 * The operation, from the pages it follows:
 *  - "Chunked prefill" (k4i.top), section "Why chunking does not change the
 *    result" (#correctness): a prompt is processed in chunks; token i of a
 *    chunk attends to every position j <= i, i.e. to the cached prefix written
 *    by earlier chunks plus the causal part of its own chunk, and the two parts
 *    combine by softmax_merge; after each chunk its new k, v vectors are
 *    appended to the KV cache.  Section "IO overhead" (#io-overhead) sizes that
 *    append: C x 2 x n_h x d_h x 2 bytes per layer.
 *  - "Disaggregated prefill and decode" (Perplexity), section "Prefill vs decode
 *    performance": decode requests carry qo_len = 1 and are memory bound,
 *    prefill requests carry large qo_len and are compute bound; attention can
 *    be split over requests and over kv_len.  Section "Sharded KV cache
 *    transfers" with the figure "NHD and HND KV cache layouts": the cache is
 *    paged in the HND layout (heads before tokens), so each head's slice of a
 *    page is contiguous.  Section "KV Messenger": KV entries are valid after
 *    the append and before attention reads them.
 *
 * Conventions shared by every call
 *  - All tensors are bf16 (bit patterns, 2 bytes per element), row-major and
 *    contiguous, on the device unless a parameter says "host".
 *  - Page pool `kv_pages`: [num_pages][2][Hkv][page_size][head_dim]; index 0 of
 *    the second dimension holds K, index 1 holds V (HND inside each page).
 *  - Page table (CSR): request r owns pages page_indices[kv_indptr[r] ..
 *    kv_indptr[r+1]); its length after this step's append is
 *    kv_len_r = (npages_r - 1) * page_size + last_page_len[r]
 *    (kv_len_r = 0 when it owns no page).  1 <= last_page_len[r] <= page_size
 *    whenever npages_r > 0.  The caller allocates pages; the table already
 *    covers the post-append length.  A page that receives appended tokens
 *    belongs to one request alone; pages that hold only cached tokens may be
 *    listed by several requests (a prefix-cache hit: "Chunked prefill",
 *    #prefix-cache-interaction), which read them in place.
 *  - Query / new-token rows (CSR): request r owns rows qo_indptr[r] ..
 *    qo_indptr[r+1]) of q, k_new, v_new and out; qo_len_r <= kv_len_r.  The new
 *    token i of request r sits at absolute position kv_len_r - qo_len_r + i.
 *  - GQA: query head h reads kv head h / (Hq / Hkv) (contiguous groups).
 *  - Ownership: the caller owns every buffer; the library allocates no device
 *    memory.  Pointers must be 16-byte aligned.
 *  - Ordering: work is enqueued on `stream` (a cudaStream_t; NULL = legacy
 *    default stream) and runs asynchronously; call daa_kv_append before
 *    daa_batch_attention on the same stream.  No call synchronises the device.
 *  - Errors: argument checks run on the host before anything is enqueued and
 *    return a negative daa_status; nothing is thrown across the ABI.  Device
 *    kernels never read or write outside the pool or the given arrays: a page
 *    id outside [0, num_pages) or an inconsistent length seen on the device is
 *    skipped and recorded in a device error word (daa_device_error).
 *  - Supported: head_dim in {64, 128}; page_size 16; 1 <= Hq/Hkv <= 16 with Hq
 *    divisible by Hkv.  Other shapes return DAA_ERR_UNSUPPORTED.
 */
#ifndef DAA_H_
#define DAA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  DAA_OK = 0,
  DAA_ERR_INVALID_ARG = -1, /* null pointer, negative count, bad scalar */
  DAA_ERR_SHAPE = -2,       /* indptr not monotonic, qo_len > kv_len, bad last_page_len */
  DAA_ERR_PAGE_RANGE = -3,  /* page count inconsistent with the pool */
  DAA_ERR_UNSUPPORTED = -4, /* head_dim / page_size / group size outside the support matrix */
  DAA_ERR_CUDA = -5,        /* a CUDA runtime call or launch failed */
  DAA_ERR_WORKSPACE = -6,   /* workspace missing or smaller than the size query */
  DAA_ERR_ALIGNMENT = -7    /* a pointer is not 16-byte aligned */
} daa_status;

typedef struct {
  int32_t num_qo_heads; /* Hq */
  int32_t num_kv_heads; /* Hkv */
  int32_t head_dim;     /* d */
  int32_t page_size;    /* P (tokens per page) */
  int64_t num_pages;    /* pages in the pool */
} daa_dims;

/* Human-readable name of a status code (static storage). */
const char* daa_status_string(daa_status s);

/* Library ABI version (major * 10000 + minor * 100 + patch). */
int32_t daa_version(void);

/*
 * KV append ("Chunked prefill", #correctness: K_cache += [k_{(s-1)C+1} .. k_{sC}];
 * #io-overhead for its size).
 *
 * For every request r and each of its n_r = append_indptr[r+1] - append_indptr[r]
 * new tokens t (0 <= t < n_r), writes
 *   kv_pages[p][0][h][s][:] = k_new[append_indptr[r] + t][h][:]
 *   kv_pages[p][1][h][s][:] = v_new[append_indptr[r] + t][h][:]
 * for every kv head h, where pos = kv_len_r - n_r + t,
 * p = page_indices[kv_indptr[r] + pos / page_size] and s = pos % page_size.
 * A bit-exact copy; nothing else in the pool is touched.
 *
 *  k_new, v_new   device, bf16 [nnz_new][Hkv][head_dim]
 *  kv_pages       device, bf16 pool (see conventions), written
 *  append_indptr  device, int32 [batch + 1], append_indptr[batch] == nnz_new
 *                 (the same array as qo_indptr of the attention call)
 *  page_indices   device, int32 [kv_indptr[batch]]
 *  kv_indptr      device, int32 [batch + 1]
 *  last_page_len  device, int32 [batch], post-append
 *  batch, nnz_new host scalars (batch >= 0, nnz_new >= 0)
 *  dims           shapes; num_qo_heads is not used here but must be valid
 *  stream         cudaStream_t
 * Errors: DAA_ERR_INVALID_ARG / _UNSUPPORTED / _ALIGNMENT on the host,
 * DAA_ERR_CUDA if the launch fails.  Lengths and page ids are checked on the
 * device (see daa_device_error).
 */
daa_status daa_kv_append(const void* k_new, const void* v_new, void* kv_pages,
                         const int32_t* append_indptr, const int32_t* page_indices,
                         const int32_t* kv_indptr, const int32_t* last_page_len, int32_t batch,
                         int32_t nnz_new, daa_dims dims, void* stream);

/*
 * Bytes of device workspace daa_batch_attention needs for this batch (0 if
 * none).  Reads the host mirrors only; a pure function of its arguments and of
 * the current device's SM count.  Returns 0 and sets *status (if non-NULL) to
 * an error for invalid input.
 */
size_t daa_batch_attention_workspace_size(const int32_t* h_qo_indptr, const int32_t* h_kv_indptr,
                                          const int32_t* h_last_page_len, int32_t batch,
                                          daa_dims dims, daa_status* status);

/*
 * Mixed-batch paged attention ("Chunked prefill", #correctness; "Disaggregated
 * prefill and decode", "Prefill vs decode performance").
 *
 * For every request r, new token i and query head h (kv head hk = h / (Hq/Hkv)),
 * with pos = kv_len_r - qo_len_r + i and key range J = {j : j <= pos} when
 * causal (J = {j < kv_len_r} otherwise):
 *   s_j = sm_scale * q[row][h][:] . K_r[j][hk][:]
 *   out[row][h][:] = sum_{j in J} softmax_J(s)_j * V_r[j][hk][:]      (bf16, RNE)
 *   lse_out[row][h] = ln sum_{j in J} exp(s_j)                          (fp32)
 * where row = qo_indptr[r] + i and K_r / V_r are read from the request's pages.
 * Routing (results do not depend on it): requests with qo_len = 1 run a
 * split-KV decode kernel (CUDA cores when a kv head serves fewer than 4 query
 * heads, tensor cores otherwise); requests with 2 <= qo_len <= min(16, 128 / g)
 * (g = Hq / Hkv; e.g. speculative-decoding verify steps) run as key-split
 * items of the tensor-core decode kernel; requests up to 256 / g tokens (two
 * 128-row tiles of packed query rows) run as items of the single-CTA
 * tensor-core kernel, key-split when long; longer requests run the
 * tensor-core prefill kernel.  Split requests are combined by the softmax_merge pass, one
 * merge per token.  Rows of requests with qo_len = 0 do not exist; nothing is
 * written.
 *
 *  q              device, bf16 [nnz_qo][Hq][head_dim]
 *  kv_pages       device, bf16 pool (read only)
 *  qo_indptr, kv_indptr, page_indices, last_page_len    device int32 (as above)
 *  h_qo_indptr, h_kv_indptr, h_last_page_len            host int32 copies of
 *                 the same arrays; used to validate and to plan the split of the
 *                 work on the host, so the call never waits on the device
 *  batch          number of requests
 *  causal         1: keys j <= pos; 0: all kv_len keys
 *  sm_scale       score scale, e.g. 1/sqrt(head_dim); must be finite and > 0
 *  out            device, bf16 [nnz_qo][Hq][head_dim], written
 *  lse_out        device, fp32 [nnz_qo][Hq] natural-log LSE, or NULL
 *  workspace      device scratch of at least
 *                 daa_batch_attention_workspace_size(...) bytes (NULL if 0);
 *                 the call owns it until the enqueued work completes
 *  stream         cudaStream_t
 * Errors: DAA_ERR_* on the host before any launch; DAA_ERR_CUDA on a failed
 * launch or copy.
 */
daa_status daa_batch_attention(const void* q, const void* kv_pages, const int32_t* qo_indptr,
                               const int32_t* kv_indptr, const int32_t* page_indices,
                               const int32_t* last_page_len, const int32_t* h_qo_indptr,
                               const int32_t* h_kv_indptr, const int32_t* h_last_page_len,
                               int32_t batch, int32_t causal, float sm_scale, void* out,
                               float* lse_out, void* workspace, size_t workspace_bytes,
                               daa_dims dims, void* stream);

/*
 * daa_kv_append followed by daa_batch_attention in one call, on one plan
 * ("Disaggregated prefill and decode", section "KV Messenger": entries are
 * valid after the append and before attention; "Chunked prefill", #correctness:
 * each chunk's new k, v are appended and attended to in the same step).
 *
 * The new tokens of request r are its query rows: k_new, v_new are
 * [nnz_qo][Hkv][head_dim] with the row layout of q (append_indptr = qo_indptr,
 * nnz_new = h_qo_indptr[batch]).  The result -- pool bytes, out, lse_out -- is
 * exactly that of the two calls in sequence on the same stream.  What differs
 * is the schedule: the plan copy is issued before the append, and the
 * attention kernels are launched behind the append as programmatic dependent
 * launches, so their set-up and the key splits that read only cached rows
 * overlap the append (the CTAs that read an appended row wait for it).
 *
 * The append of long prefill chunks is fused into their attention ("Chunked
 * prefill", #io-overhead: the chunk's K/V are written to the cache once).  A
 * request with more new tokens than two 128-row tiles of packed (token, query
 * head) rows hold (qo_len > 2 * (128 / (Hq / Hkv))) runs on a prefill kernel
 * (CTA pairs for head_dim 128, one CTA per two tiles for head_dim 64).  Its
 * key tiles that lie wholly in the chunk -- keys from the first multiple of 128
 * at or after kv_len - qo_len -- are read by that kernel straight from k_new /
 * v_new, and written into their pages by it from the same tiles; the append
 * kernel writes only the other rows.  The pages end up with exactly the bytes
 * the plain append writes.
 * daa_set_prefill_append_fusion(0) turns this off (every row then goes
 * through the append kernel and is read back from the pages).
 *
 *  k_new, v_new   device, bf16 [nnz_qo][Hkv][head_dim]
 *  kv_pages       device, bf16 pool, written (the appended rows) and read
 *  other arguments as daa_batch_attention, with the same workspace size
 *  (daa_batch_attention_workspace_size).
 * Errors: those of both calls, all checked on the host before anything is
 * enqueued.
 */
daa_status daa_append_attention(const void* k_new, const void* v_new, const void* q,
                                void* kv_pages, const int32_t* qo_indptr,
                                const int32_t* kv_indptr, const int32_t* page_indices,
                                const int32_t* last_page_len, const int32_t* h_qo_indptr,
                                const int32_t* h_kv_indptr, const int32_t* h_last_page_len,
                                int32_t batch, int32_t causal, float sm_scale, void* out,
                                float* lse_out, void* workspace, size_t workspace_bytes,
                                daa_dims dims, void* stream);

/*
 * One serving step fed from host memory: upload the step's inputs, run
 * daa_append_attention on them, read the output back -- one call per step,
 * every copy and kernel asynchronous, so consecutive steps overlap when the
 * caller alternates two sets of device buffers.  It feeds the attention and
 * the append as a serving loop does ("Accelerating Sonar through
 * speculation", section "Inference with speculative decoding": a step's input
 * tokens and KV page information are packed into one buffer on the host and
 * the metadata is then copied to GPU memory).
 *
 * Inputs: one pinned host buffer `h_inputs` of layout->total bytes holding,
 * at the byte offsets of `layout`, the step's qo_indptr, kv_indptr,
 * page_indices, last_page_len (int32, 4-byte aligned offsets) and q, k_new,
 * v_new (bf16, 16-byte aligned offsets), with the shapes of
 * daa_append_attention.  The call reads the page table from this host buffer
 * to plan (no device sync), copies the whole buffer to `d_inputs` (device,
 * 256-byte aligned, layout->total bytes) on the upload stream, runs the append
 * and the attention on the compute stream from the device copy, and copies
 * out ([nnz_qo][Hq][head_dim] bf16 in `d_out`) back to `h_out` (pinned host)
 * on the download stream.  `workspace` is that of daa_append_attention.
 *
 * Ordering (all cudaEvent_t / cudaStream_t, created by the caller):
 *   upload:   waits for streams->inputs_free (if not NULL: the previous step
 *             that read this d_inputs has finished computing), copies, records
 *             streams->uploaded;
 *   compute:  waits for uploaded and for streams->out_free (if not NULL: the
 *             previous read-back of this d_out has finished), runs the kernels,
 *             records streams->computed;
 *   download: waits for computed, copies, records streams->downloaded.
 * h_inputs must not change until `uploaded` has completed; h_out holds the
 * output once `downloaded` has completed.  A batch with no query rows copies
 * nothing and only records the three events.
 *
 * Errors: those of daa_append_attention, plus DAA_ERR_INVALID_ARG for a NULL
 * buffer, layout, stream set or event, DAA_ERR_ALIGNMENT for misaligned
 * offsets or d_inputs, DAA_ERR_SHAPE when a section runs past layout->total.
 * All are found before anything is enqueued.
 */
typedef struct {
  size_t qo_indptr, kv_indptr, page_indices, last_page_len; /* int32 sections */
  size_t q, k_new, v_new;                                   /* bf16 sections */
  size_t total;                                             /* bytes uploaded */
} daa_step_layout;

typedef struct {
  void* upload_stream;   /* cudaStream_t */
  void* compute_stream;  /* cudaStream_t */
  void* download_stream; /* cudaStream_t */
  void* uploaded;        /* cudaEvent_t, recorded by the call */
  void* computed;        /* cudaEvent_t, recorded by the call */
  void* downloaded;      /* cudaEvent_t, recorded by the call */
  void* inputs_free;     /* cudaEvent_t waited for, or NULL */
  void* out_free;        /* cudaEvent_t waited for, or NULL */
} daa_step_streams;

daa_status daa_append_attention_host(const void* h_inputs, void* d_inputs,
                                     const daa_step_layout* layout, int32_t batch, int32_t causal,
                                     float sm_scale, void* kv_pages, void* d_out, void* h_out,
                                     void* workspace, size_t workspace_bytes, daa_dims dims,
                                     const daa_step_streams* streams);

/*
 * Switch of the fused prefill append of daa_append_attention,
 * daa_append_attention_shared_prefix and daa_append_attention_run ("Chunked
 * prefill", #io-overhead; see daa_append_attention): 1 (the default) lets the
 * prefill kernels read their chunk's own key tiles from k_new / v_new and
 * write them into the pages; 0 appends every row with the append kernel.
 * Results (pool bytes, out, lse_out) are identical; only the work differs.
 * Process-wide; takes effect for calls made after it returns.
 * Errors: DAA_ERR_INVALID_ARG for a value other than 0 or 1.
 */
daa_status daa_set_prefill_append_fusion(int32_t enable);

/* The current setting of daa_set_prefill_append_fusion (0 or 1). */
int32_t daa_prefill_append_fusion(void);

/*
 * Mixed-batch paged attention under draft-tree masks, for verifying the draft
 * tokens of speculative decoding ("Accelerating Sonar through speculation"
 * (Perplexity), section EAGLE: a tree of draft tokens is checked by the target
 * model in one pass under a custom attention mask; each draft token is scored
 * against the accepted prefix and its own branch of the tree).
 *
 * Computes daa_batch_attention with causal = 1, except that new token i of a
 * request sees, among the request's new tokens, only itself and the earlier
 * ones its mask row selects.  With pos0 = kv_len - qo_len (the key of new token
 * 0), token i's key set is
 *   J = {j < pos0}  U  {pos0 + i}  U  {pos0 + t : t < i, bit t of its row set}.
 * Mask rows: tree_mask is uint32 [nnz_qo][mask_words] on the device, one row
 * per query row (the row layout of q); bit t of a row is word t / 32, bit
 * t % 32 (t counts the request's new tokens from 0).  Bits t >= i are ignored:
 * a token always sees itself and never a later new token, so a row of all
 * earlier bits set is plain causal attention and every request of a mixed
 * batch can be given that way.  For a draft tree whose nodes are numbered so
 * that parents precede children, row i holds the bits of i's ancestors.
 * Requests with qo_len = 1 are unaffected (their key set is the same).
 *
 *  tree_mask      device, uint32 [nnz_qo][mask_words], 4-byte aligned
 *  mask_words     words per row; every request needs qo_len <= 32 * mask_words
 *  other arguments as daa_batch_attention (no `causal`: the rule is causal),
 *  with the same workspace size (daa_batch_attention_workspace_size).
 * Errors: those of daa_batch_attention; DAA_ERR_INVALID_ARG for a NULL mask or
 * mask_words < 1, DAA_ERR_SHAPE when a request has more than 32 * mask_words
 * new tokens, DAA_ERR_ALIGNMENT for a misaligned mask.  Only tiles of keys
 * that hold earlier new tokens of a row evaluate the mask; the cached prefix
 * streams exactly as in daa_batch_attention.
 */
daa_status daa_batch_attention_tree(const void* q, const void* kv_pages,
                                    const int32_t* qo_indptr, const int32_t* kv_indptr,
                                    const int32_t* page_indices, const int32_t* last_page_len,
                                    const int32_t* h_qo_indptr, const int32_t* h_kv_indptr,
                                    const int32_t* h_last_page_len, int32_t batch,
                                    const uint32_t* tree_mask, int32_t mask_words, float sm_scale,
                                    void* out, float* lse_out, void* workspace,
                                    size_t workspace_bytes, daa_dims dims, void* stream);

/*
 * Mixed-batch paged attention for requests that share a cached prefix, with
 * that prefix's keys read once for the whole group ("Chunked prefill"
 * (k4i.top), #prefix-cache-interaction: the cached blocks of a prefix hit are
 * skipped, only the suffix is computed; #correctness: attention over a key set
 * is the softmax_merge of attentions over a partition of it).
 *
 * The result -- out, lse_out -- is that of daa_batch_attention on the same
 * arguments (equal up to fp32 rounding order).  What differs is the schedule.
 * Within a group, every run of consecutive decode, verify and short requests
 * (1 <= qo_len <= two 128-row Q tiles of packed (token, head) rows) with two
 * or more such members has the query rows of all its members (one per new
 * token and query head) attended to the group's shared keys in one pass, the
 * rows of several requests packed into the same 128-row tensor-core tiles.
 * Only whole 128-key tiles of the prefix are shared; the rest of it is read
 * per request.  Each member's own items then cover only the keys after the
 * shared part, and softmax_merge combines the two parts per row.  K/V bytes of
 * the shared prefix are read once per run instead of once per request.
 * Prefill requests of a group (and runs of one member) attend the prefix in
 * their own items: their Q tiles are full already.
 *
 * Groups (host arrays): group i is requests [h_prefix_indptr[i],
 * h_prefix_indptr[i+1]) -- consecutive requests, groups in request order --
 * whose first h_prefix_len[i] keys are the same tokens in the same pages: for
 * every request r of the group, page_indices[kv_indptr[r] + p] is the same
 * page for every p < h_prefix_len[i] / page_size.  The library cannot check
 * this (page ids live only on the device); a group that breaks it gives wrong
 * outputs, never an access outside the pool.  h_prefix_len[i] must be a
 * multiple of page_size and cached: at most kv_len_r - qo_len_r for every
 * request of the group.  Requests in no group are planned as in
 * daa_batch_attention; a request between two groups may sit in a group of
 * prefix length 0.
 *
 *  h_prefix_indptr  host int32 [n_groups + 1], non-decreasing, in [0, batch]
 *  h_prefix_len     host int32 [n_groups]
 *  n_groups         >= 0 (0: exactly daa_batch_attention's plan)
 *  workspace        at least daa_batch_attention_shared_prefix_workspace_size(...)
 *                   bytes with the same groups
 *  other arguments as daa_batch_attention / daa_append_attention.
 * Errors: those of daa_batch_attention; DAA_ERR_INVALID_ARG for n_groups < 0
 * or NULL group arrays with n_groups > 0; DAA_ERR_SHAPE for a group outside
 * [0, batch], a decreasing indptr, a prefix length that is negative, not a
 * multiple of page_size, or longer than some member's cached keys.
 */
size_t daa_batch_attention_shared_prefix_workspace_size(
    const int32_t* h_qo_indptr, const int32_t* h_kv_indptr, const int32_t* h_last_page_len,
    int32_t batch, const int32_t* h_prefix_indptr, const int32_t* h_prefix_len, int32_t n_groups,
    daa_dims dims, daa_status* status);

daa_status daa_batch_attention_shared_prefix(
    const void* q, const void* kv_pages, const int32_t* qo_indptr, const int32_t* kv_indptr,
    const int32_t* page_indices, const int32_t* last_page_len, const int32_t* h_qo_indptr,
    const int32_t* h_kv_indptr, const int32_t* h_last_page_len, int32_t batch,
    const int32_t* h_prefix_indptr, const int32_t* h_prefix_len, int32_t n_groups, int32_t causal,
    float sm_scale, void* out, float* lse_out, void* workspace, size_t workspace_bytes,
    daa_dims dims, void* stream);

/* daa_append_attention (append, then attention, in one call) with the prefix
 * groups of daa_batch_attention_shared_prefix. */
daa_status daa_append_attention_shared_prefix(
    const void* k_new, const void* v_new, const void* q, void* kv_pages, const int32_t* qo_indptr,
    const int32_t* kv_indptr, const int32_t* page_indices, const int32_t* last_page_len,
    const int32_t* h_qo_indptr, const int32_t* h_kv_indptr, const int32_t* h_last_page_len,
    int32_t batch, const int32_t* h_prefix_indptr, const int32_t* h_prefix_len, int32_t n_groups,
    int32_t causal, float sm_scale, void* out, float* lse_out, void* workspace,
    size_t workspace_bytes, daa_dims dims, void* stream);

/*
 * Plan once, run many times.  The plan of a batch -- how its requests are cut
 * into work items ("Disaggregated prefill and decode", "Prefill vs decode
 * performance": attention splits over requests and over kv_len) -- depends
 * only on the page table's lengths.  In a model, every attention layer of a
 * step reads the same table, so one plan serves all of them.
 * daa_batch_attention_plan builds it on the host and copies it into the head
 * of the workspace (one cudaMemcpyAsync on `stream`).  daa_batch_attention_run
 * and daa_append_attention_run then launch only the kernels.  The outputs are
 * bit-identical to daa_batch_attention / daa_append_attention on the same
 * arguments, with and without prefix groups.
 *
 * daa_plan_info is plain data: the workspace layout and the shapes the plan
 * was made for.  The plan stays valid while the workspace is not written by
 * anything else (another plan, or a call that plans for itself) and the page
 * table's lengths (qo_indptr, kv_indptr, last_page_len) are unchanged.  The
 * pages themselves and q, k_new, v_new may change between runs.  Runs of one
 * plan must not overlap on the GPU: they share the workspace's partials.
 *
 *  plan: the host arrays of daa_batch_attention (plus the prefix groups of
 *        daa_batch_attention_shared_prefix; n_groups = 0 for none), the
 *        workspace (at least the matching workspace-size query's bytes; may be
 *        NULL when that size is 0), `info` (written), `stream`.
 *  run:  the device arrays of daa_batch_attention, `info`, then causal,
 *        sm_scale, out, lse_out, the workspace, the dims the plan was made
 *        for, `stream`.  The page table passed must be the one planned.
 * Errors: plan -- those of the size query; DAA_ERR_INVALID_ARG for a NULL info;
 * DAA_ERR_WORKSPACE / DAA_ERR_ALIGNMENT for the workspace; DAA_ERR_CUDA if the
 * copy fails.  run -- DAA_ERR_INVALID_ARG for an info that no plan call wrote or
 * whose dims differ from `dims`; otherwise those of daa_batch_attention.
 */
typedef struct {
  int64_t words[24];
} daa_plan_info;

daa_status daa_batch_attention_plan(const int32_t* h_qo_indptr, const int32_t* h_kv_indptr,
                                    const int32_t* h_last_page_len, int32_t batch,
                                    const int32_t* h_prefix_indptr, const int32_t* h_prefix_len,
                                    int32_t n_groups, daa_dims dims, void* workspace,
                                    size_t workspace_bytes, daa_plan_info* info, void* stream);

daa_status daa_batch_attention_run(const void* q, const void* kv_pages, const int32_t* qo_indptr,
                                   const int32_t* kv_indptr, const int32_t* page_indices,
                                   const int32_t* last_page_len, const daa_plan_info* info,
                                   int32_t causal, float sm_scale, void* out, float* lse_out,
                                   void* workspace, size_t workspace_bytes, daa_dims dims,
                                   void* stream);

/* daa_append_attention on a plan: the append of k_new, v_new, then the
 * attention kernels launched behind it (as daa_append_attention). */
daa_status daa_append_attention_run(const void* k_new, const void* v_new, const void* q,
                                    void* kv_pages, const int32_t* qo_indptr,
                                    const int32_t* kv_indptr, const int32_t* page_indices,
                                    const int32_t* last_page_len, const daa_plan_info* info,
                                    int32_t causal, float sm_scale, void* out, float* lse_out,
                                    void* workspace, size_t workspace_bytes, daa_dims dims,
                                    void* stream);

/* Size of the device scratch array behind daa_batch_attention_noalloc (48 MiB). */
#define DAA_NOALLOC_SCRATCH_BYTES (48u * 1024u * 1024u)

/*
 * daa_batch_attention for callers that cannot allocate device memory.  The
 * pages describe no such call; it has no counterpart there.
 *
 * Who needs it: a caller with no device allocator at the call site -- e.g. a
 * serving engine that has handed all free HBM to its KV page pool and keeps no
 * allocator to carve a workspace from, code on a latency-critical path where a
 * cudaMalloc/cudaFree could synchronise the device, or a foreign-language host
 * with no binding to a CUDA allocator.  It computes exactly what
 * daa_batch_attention computes, with the same arguments minus the workspace.
 *
 * Scratch: the work plan and the split-KV partial outputs live in one
 * file-scope __device__ array of DAA_NOALLOC_SCRATCH_BYTES bytes, which every
 * GPU that loads the library holds until the process exits.  The call makes no
 * cudaMalloc/cudaFree and no other allocation (device or host heap); its plan
 * is built in fixed-size static host buffers.  A batch whose scratch would
 * exceed the array, or that needs more than 16384 decode splits, 16384 split
 * requests or 16384 prefill tiles, is rejected with DAA_ERR_WORKSPACE before
 * anything is enqueued.
 *
 * Set-up: the first call on each device (with that device current) looks up
 * the array's device address with cudaGetSymbolAddress and caches it.  The
 * cached address belongs to the device context it was looked up in: after
 * cudaDeviceReset (or anything else that destroys the primary context) it is
 * stale, so do not call this entry point again in a process that has reset the
 * device.
 *
 * Sharing: every call, on every stream and host thread, uses the same array,
 * which keeps the last call's contents.  Nothing in it has to start at zero --
 * every byte a call reads was written earlier in that same call -- but calls
 * whose GPU work overlaps (concurrent streams, or calls from several host
 * threads without ordering between their streams) race on the scratch and
 * produce wrong results.  Serialise them, e.g. by issuing all such calls on one
 * stream.  Host-side calls are serialised by an internal mutex.
 *
 * Arguments, layouts and the other errors are those of daa_batch_attention.
 */
daa_status daa_batch_attention_noalloc(const void* q, const void* kv_pages,
                                       const int32_t* qo_indptr, const int32_t* kv_indptr,
                                       const int32_t* page_indices, const int32_t* last_page_len,
                                       const int32_t* h_qo_indptr, const int32_t* h_kv_indptr,
                                       const int32_t* h_last_page_len, int32_t batch,
                                       int32_t causal, float sm_scale, void* out, float* lse_out,
                                       daa_dims dims, void* stream);

/*
 * Step tables built on the GPU ("Accelerating Sonar through speculation", section
 * "Inference with speculative decoding": the KV page information of a step is
 * metadata that the attention kernel is configured with; "Disaggregated prefill
 * and decode", section "KV Messenger": pages are allocated per request).
 *
 * daa_page_pool holds the pages of many requests on the device, one slot each.
 * All arrays belong to the caller:
 *   seq_len      int32 [num_slots]             cached tokens of the slot
 *   held         int32 [num_slots]             pages in the slot's row
 *   block_table  int32 [num_slots][max_pages]  their ids, in token order
 *   free_pages   int32 [num_pages]             a stack; entries [0, counters[0])
 *   counters     int32 [2]                     free pages; scratch (0 before the
 *                                              first call, and 0 after each)
 * held may be more than seq_len needs (a request cut back after rejected draft
 * tokens keeps its pages and uses them again).
 *
 * daa_step_table: for a step that brings new_len[i] >= 0 tokens to slot slots[i],
 * with kv_i = seq_len + new_len[i] and n_i = ceil(kv_i / page_size),
 *   qo_indptr, kv_indptr   int32 [batch + 1]: exclusive sums of new_len and n_i
 *   page_indices           int32 [page_capacity]: the n_i pages of each request;
 *                          entries past kv_indptr[batch] are left as they were
 *   last_page_len          int32 [batch]: kv_i - (n_i - 1) * page_size (0 if n_i = 0)
 *   slot_map               int64 [row_capacity] or NULL: page * page_size + slot of
 *                          every new token (its place in the pool), in row order
 *   positions              int32 [row_capacity] or NULL: seq_len + j of new token j
 * -- the page table of this header's other calls.  Pages a request lacks come
 * from the top of the free stack, in request order, and are added to its row;
 * held and the free count follow.  seq_len is advanced by new_len when `advance`
 * is 1; with 0 it stays, and the same call can be made again (it then takes no
 * pages), for callers that learn how many tokens were accepted afterwards.
 *
 * All or nothing: if a slot is out of range or named twice, new_len < 0, kv_i >
 * max_pages * page_size, the capacities are too small, or the stack holds too
 * few pages, the pool is not changed, both indptr arrays and last_page_len are
 * zero (an empty step), and the device error word is set (3, or 4 for too few
 * free pages).
 *
 * daa_release_pages: the pages of `batch` slots go back on the stack; their
 * seq_len and held become 0.  Nothing is changed if a slot is out of range or
 * named twice, or the stack has no room (error word 3).
 *
 * Calls on one pool must not overlap on the GPU (they share its counters).  One
 * kernel launch each, no host copies: both can be captured into a CUDA graph.
 * Errors (host): DAA_ERR_INVALID_ARG for NULL arrays, negative counts or advance
 * not 0 or 1; DAA_ERR_UNSUPPORTED for page_size != 16, batch >
 * DAA_STEP_MAX_BATCH, num_slots > DAA_STEP_MAX_SLOTS; DAA_ERR_ALIGNMENT for a
 * slot_map that is not 8-byte aligned; DAA_ERR_CUDA for a failed launch.
 */
#define DAA_STEP_MAX_BATCH 8192
#define DAA_STEP_MAX_SLOTS 65536

typedef struct {
  int32_t* seq_len;
  int32_t* held;
  int32_t* block_table;
  int32_t* free_pages;
  int32_t* counters;
  int32_t num_slots;
  int32_t max_pages; /* pages of a row */
  int32_t num_pages; /* entries of the stack */
  int32_t page_size; /* 16 */
} daa_page_pool;

daa_status daa_step_table(const daa_page_pool* pool, const int32_t* slots, const int32_t* new_len,
                          int32_t batch, int32_t advance, int32_t* qo_indptr, int32_t* kv_indptr,
                          int32_t* page_indices, int32_t page_capacity, int32_t* last_page_len,
                          int64_t* slot_map, int32_t* positions, int32_t row_capacity,
                          void* stream);

daa_status daa_release_pages(const daa_page_pool* pool, const int32_t* slots, int32_t batch,
                             void* stream);

/*
 * The 4-bit KV cache.  Decode attention is bound by the K/V bytes it reads
 * ("Disaggregated prefill and decode", "Prefill vs decode performance"); this
 * cache holds 4.5 bits a value instead of 16.
 *
 * Format.  A value is e2m1 * e4m3 * 2^e: a 4-bit float (values 0, .5, 1, 1.5, 2,
 * 3, 4, 6 and their negatives, codes 0..7 and 8..15), the e4m3 scale of its
 * block of 16 dims of one token and kv head, and the exponent of its kv head.
 * Pool: uint8 [num_pages][Hkv][2 (K, V)][9 * head_dim] -- heads before tokens, as
 * the bf16 pool, with a head's K and V of a page side by side.  A slice holds
 *   16 token rows of head_dim / 2 bytes: dim 2i in the low four bits of byte i,
 *   dim 2i + 1 in the high four; then head_dim scale bytes:
 *   K: [16 tokens][head_dim / 16 blocks],  V: [head_dim / 16 blocks][16 tokens].
 * kv_exp: int32 [2 (K, V)][Hkv] on the device, or NULL for zeros; read as at
 * least -32 and at most 32.  The same exponents go to every call on a pool.
 * They centre a head's values in the range of its scales (2^-9 .. 448).
 *
 * daa_kv_append_q4: daa_kv_append into a 4-bit pool (same arguments, checks and
 * errors).  For a block x of 16 bf16 values, y = x * 2^-e:
 *   scale = e4m3(clamp(max|y| / 6, 2^-9, 448)), code = e2m1(y / scale),
 * each rounded to the nearest value, ties to the even code, cut at 6; a zero
 * keeps its sign bit.  NaN is stored as zero and an infinity as +-6 * 448 * 2^e,
 * so the cache holds finite values only.  Only the new tokens' bytes are written.
 *
 * daa_kv_dequant_q4: pages page_ids[0 .. n_pages) (device int32) as bf16 pages
 * out[i][2][Hkv][16][head_dim], exactly (a value has at most 6 significant bits).
 * A page id outside [0, num_pages) gives a page of zeros and sets the device
 * error word (1).  Errors as daa_kv_append.
 *
 * daa_batch_attention_q4_*: daa_batch_attention over a 4-bit pool, planned once
 * and run many times (see daa_batch_attention_plan and _run: same plan rules,
 * workspace, causal mask, outputs and errors).  Draft-tree masks and shared-prefix
 * groups have no form of this; daa_kv_dequant_q4 gives pages that the bf16 calls
 * take.  The result is that of daa_batch_attention on the pool's values in bf16,
 * up to fp32 rounding order and the rounding of the softmax weights.  Slots past a
 * request's last token may hold anything.
 * Requests of up to 96 packed (token, query head) rows are read from the 4-bit
 * pages, with weights rounded to fp16 (2^-11 of a weight), and so are longer
 * chunks where a batch has few of them.  The pages of the other chunks are written
 * to the workspace in bf16 by every run (2 * Hkv * head_dim * 32 bytes a page; a
 * page that two such requests share is written for each), and their weights are
 * rounded to bf16 (2^-8).  The plan decides from the whole batch, so a chunk's last
 * bits may depend on what else is in it.
 * What the cache gains is decode and verify speed: from about 64 rows a request on,
 * a batch of many requests is slower than daa_batch_attention on bf16 pages
 * (GB300, 32 requests of 2500 keys, 8 kv heads of 128 dims: 25.7 us and 62.2 at 4
 * rows, 65 and 68 at 48, 91 and 71 at 64, 118 and 66 to 77 at 96, 150 and 83 at 256).
 * Scores are fp32: a row with a scaled score past 2^26 in magnitude is undefined.
 *  plan: host arrays of daa_batch_attention; the workspace (at least
 *        daa_batch_attention_q4_workspace_size bytes, 256-byte aligned); `info`.
 *        It copies from host memory, so it cannot be captured into a CUDA graph
 *        (DAA_ERR_UNSUPPORTED on a capturing stream); run can.
 *  run:  q, out [nnz_qo][Hq][head_dim] bf16, lse_out fp32 [nnz_qo][Hq] or NULL,
 *        page_indices (device) of the planned table.
 * Runs that share a workspace must not overlap on the GPU, whatever stream or
 * graph they are launched from.
 */
daa_status daa_kv_append_q4(const void* k_new, const void* v_new, void* kv_pages,
                            const int32_t* kv_exp, const int32_t* append_indptr,
                            const int32_t* page_indices, const int32_t* kv_indptr,
                            const int32_t* last_page_len, int32_t batch, int32_t nnz_new,
                            daa_dims dims, void* stream);

daa_status daa_kv_dequant_q4(const void* kv_pages, const int32_t* kv_exp, const int32_t* page_ids,
                             int32_t n_pages, void* out, daa_dims dims, void* stream);

size_t daa_batch_attention_q4_workspace_size(const int32_t* h_qo_indptr, const int32_t* h_kv_indptr,
                                             const int32_t* h_last_page_len, int32_t batch,
                                             daa_dims dims, daa_status* status);

daa_status daa_batch_attention_q4_plan(const int32_t* h_qo_indptr, const int32_t* h_kv_indptr,
                                       const int32_t* h_last_page_len, int32_t batch, daa_dims dims,
                                       void* workspace, size_t workspace_bytes, daa_plan_info* info,
                                       void* stream);

daa_status daa_batch_attention_q4_run(const void* q, const void* kv_pages, const int32_t* kv_exp,
                                      const int32_t* page_indices, const daa_plan_info* info,
                                      int32_t causal, float sm_scale, void* out, float* lse_out,
                                      void* workspace, size_t workspace_bytes, daa_dims dims,
                                      void* stream);

/*
 * Rotary positions ("Chunked prefill", #correctness: a chunk's new k, v vectors
 * join the cache at their absolute positions).  The other calls of this header
 * take q and k whose heads are rotated by their tokens' positions already; these
 * apply the rotation, alone or on the way into the cache.
 *
 * Of a head x[0 .. head_dim) of a token at position p, the first rotary_dim dims
 * form pairs (a, b): (x[i], x[i + rotary_dim / 2]), or (x[2i], x[2i + 1]) when
 * interleaved.  Pair i becomes
 *   m * (a cos t - b sin t, b cos t + a sin t),  t = p * radians[i],
 * and the other dims stay as they are.  With norm weights (q_norm, k_norm: bf16
 * [head_dim]) a head is first divided by sqrt(mean of its squares + eps) and
 * multiplied by the weights, all of its dims.  Computed in fp32, rounded once to
 * bf16; the angle is good to 2^-33 of a turn at every position from -2^31 to
 * 2^31 - 1.  Dims that are neither normalised nor rotated keep their bits.  (The
 * squares are summed in fp32: heads of values past about 10^18 have no norm, nor, with
 * eps 0, those of values under 10^-19.)
 * Rotating by negated positions is the transposed rotation: it takes gradients of
 * the outputs to gradients of the inputs, and for m = 1 outputs back to inputs.
 *
 * daa_rope: plain data, filled by daa_rope_init from the radians per token of each
 * of the rotary_dim / 2 pairs (a host array; whatever scaling a model uses for long
 * contexts is in them) and the magnitude m.  The calls read it on the host.
 * Errors: DAA_ERR_UNSUPPORTED for head_dim not 64 or 128, or a rotary_dim that is
 * not a multiple of 16 from 16 to head_dim; DAA_ERR_INVALID_ARG for NULL arguments,
 * interleaved not 0 or 1, a magnitude outside DAA_ROPE_MIN_MAGNITUDE ..
 * DAA_ROPE_MAX_MAGNITUDE, or |radians| that is not at most DAA_ROPE_MAX_RADIANS.
 */
#define DAA_ROPE_MAX_RADIANS 1048576.0
#define DAA_ROPE_MAX_HEADS 1073741824 /* of all rows of a call */
#define DAA_ROPE_MIN_MAGNITUDE 0.0009765625
#define DAA_ROPE_MAX_MAGNITUDE 1024.0

typedef struct {
  uint64_t turns[64]; /* of pair i: turns a token, times 2^64, modulo 2^64 */
  int32_t head_dim;
  int32_t rotary_dim;
  int32_t interleaved;
  double magnitude;
} daa_rope;

daa_status daa_rope_init(daa_rope* rope, int32_t head_dim, int32_t rotary_dim, int32_t interleaved,
                         const double* radians, double magnitude);

/* bf16 rows [num_rows][heads][head_dim] on the device: the head_dim values of a head
 * side by side, strides in elements.  q, k and v may be views of one projection's
 * output.  Addresses are 16-byte aligned, strides multiples of 8 (of a dimension of
 * one entry they are not looked at). */
typedef struct {
  void* data;
  int64_t row_stride;
  int64_t head_stride;
} daa_rows;

typedef struct {
  daa_rows q, k, v;         /* read */
  daa_rows q_out, k_out;    /* written */
  int32_t num_rows;
  const int32_t* positions; /* device, int32 [num_rows] */
  const void* q_norm;       /* device, bf16 [head_dim], or NULL: no norm */
  const void* k_norm;
  float eps;                /* finite, >= 0; read when there is a norm */
} daa_rope_rows;

/*
 * daa_apply_rope: q_out = rotated q, k_out = rotated k, by `positions`.  num_q_heads
 * >= 1, num_k_heads >= 0 (0: k and k_out are not looked at; v never is).
 *
 * daa_append_rope, daa_append_rope_q4: daa_kv_append and daa_kv_append_q4 of the
 * rotated k and of v, and q_out = rotated q, in one pass over the projections'
 * rows.  bf16 pages get exactly the bytes of daa_apply_rope followed by daa_kv_append.
 * Keys on their way to 4 bits are rotated to the nearest fp32 value, rounded to bf16
 * from that, and quantised: their codes are those of the definition, not of an order of
 * fp32 operations.  Nearest up to one in some 2^12 that lies next to the middle of two,
 * at positions within 2^24 of zero; beyond, where the angle is off by p 2^-65 turns, up
 * to twice as many with each doubling (one in some 2^6 at 2^31).  Which bf16 value it is
 * hangs on that at one in some 2^27 and 2^22.
 * Rows belong to requests by append_indptr, and a row's position is its place in
 * its request, kv_len_r - n_r + t, unless `positions` gives others (draft trees:
 * the depths; the page and slot are by its place always).  q.data NULL: there are
 * no query rows (q_out.data is NULL then); dims.num_qo_heads must be valid all the
 * same.  k_out is not looked at.  dims, kv_pages, kv_exp and the table as in the calls named.
 * num_rows may be more than append_indptr[batch]: rows behind the last request are
 * padding, and nothing is written for them (a captured step's buffers hold the
 * most rows that a step may have).
 *
 * An output may be its own input (same address and strides: in place).  Otherwise no
 * output may share an element with another output or with the rows, positions, weights
 * or tables that are read, and neither outputs nor what is read may lie in the pool:
 * what cannot be told apart by ranges, by columns of the same rows or by heads of the
 * same order is refused (of page_indices, whose number is on the device, the first).
 * One kernel launch each, no workspace, nothing kept: all can be captured into a CUDA
 * graph, and calls on different rows and pages may overlap.
 * Errors: DAA_ERR_INVALID_ARG for NULL arguments (positions of daa_apply_rope among
 * them), negative counts or strides, an eps or overlap as above, a rope of another
 * head_dim than dims; DAA_ERR_UNSUPPORTED for more than DAA_ROPE_MAX_HEADS heads of
 * all rows or requests, and shapes as daa_kv_append; DAA_ERR_SHAPE for rows without requests (batch 0);
 * DAA_ERR_ALIGNMENT; DAA_ERR_CUDA.  Lengths and page ids are checked on the device:
 * nothing is written for a row of a request with inconsistent lengths (starts below
 * zero, ends before starts or behind the last request's page, error word 3);
 * of a row whose page id is outside the pool only q_out is (error word 1).
 */
daa_status daa_apply_rope(const daa_rope* rope, const daa_rope_rows* rows, int32_t num_q_heads, int32_t num_k_heads,
                          void* stream);

daa_status daa_append_rope(const daa_rope* rope, const daa_rope_rows* rows, void* kv_pages,
                           const int32_t* append_indptr, const int32_t* page_indices, const int32_t* kv_indptr,
                           const int32_t* last_page_len, int32_t batch, daa_dims dims, void* stream);

daa_status daa_append_rope_q4(const daa_rope* rope, const daa_rope_rows* rows, void* kv_pages, const int32_t* kv_exp,
                              const int32_t* append_indptr, const int32_t* page_indices, const int32_t* kv_indptr,
                              const int32_t* last_page_len, int32_t batch, daa_dims dims, void* stream);

/*
 * Reads the device error word of the current device into *code (0 = none, 1 =
 * page id out of range, 2 = a bounded wait timed out, 3 = inconsistent request
 * lengths, 4 = a step table that needs more pages than are free) and clears it
 * when `reset` is non-zero.  Synchronises the device.
 * Kernels never trap on these: a page id outside the pool is replaced by page
 * 0 (or, in the append, the row is skipped), so the outputs of that call are
 * undefined but the context stays usable.  Every wait inside a kernel is
 * bounded (1 s); one that runs out records code 2 and the kernel runs on to its
 * exit.  While the word holds code 2, waits of later launches give up at once,
 * so clear it (reset = 1) after a timeout has been reported.
 */
daa_status daa_device_error(int32_t* code, int32_t reset);

/*
 * Health check of the bounded waits (no counterpart on the pages): launches a
 * one-thread kernel on the legacy default stream that waits on an mbarrier
 * phase nothing completes, with the same bounded wait the attention kernels
 * use, and returns after that wait has given up (about 1 s).  *gave_up = 1 when
 * the wait ended by its limit; the device error word then holds code 2 (read
 * and clear it with daa_device_error).  Synchronises the device.
 */
daa_status daa_selftest_bounded_wait(int32_t* gave_up);

/*
 * Per-kernel timing with CUDA events.  While enabled, every kernel the library
 * launches is bracketed by two events on its stream (up to `capacity` launches
 * are kept, older ones dropped).  daa_trace_read synchronises on the recorded
 * events and copies out up to `max_records` (kernel id, milliseconds) pairs in
 * launch order, returning how many were written, then clears the record.
 * Kernel ids: 1 kv_append, 2 decode split-KV (CUDA cores), 3 softmax_merge,
 * 4 tensor-core prefill, 5 tensor-core decode split-KV (decode and verify
 * items), 6 tensor-core short multi-token items (head_dim 128: requests whose
 * rows fit two 128-row Q tiles), 7 step tables and released pages, 8 4-bit
 * append, 9 4-bit pages to bf16, 10 attention over 4-bit pages, 11 rotated rows,
 * 12 and 13 the append with rotation into bf16 and 4-bit pages.
 */
daa_status daa_trace_enable(int32_t capacity);
daa_status daa_trace_disable(void);
int32_t daa_trace_read(int32_t* kernel_ids, float* milliseconds, int32_t max_records);

#ifdef __cplusplus
}
#endif

#endif /* DAA_H_ */
