/*
 * sdpa.h — C ABI of a fused, memory-efficient scaled-dot-product attention
 * forward pass for NVIDIA GB300 (sm_103a).
 *
 *   O   = softmax(scale * Q K^T + mask [+ sink column]) V
 *   LSE = ln( sum_j exp(scale * q.k_j + mask_j) [+ exp(sink)] )
 *
 * The operation is the one named by the problem statement of MLX PR #964
 * ("Metal shaders for memory efficient self attention on large sequences",
 * the call mx.fast.scaled_dot_product_attention(queries, keys, values,
 * scale=scale, mask=None)) widened by MLX PR #4459 ("Add D512 support to
 * Metal vector attention": grouped-query heads, head_dim 512, per-head
 * sinks, single-query decode through single-pass and two-pass vector
 * kernels) and by the option set of the cuDNN graph built in mlx 0.30.7
 * mlx/backend/cuda/scaled_dot_product_attention.cpp (build_sdpa_graph:
 * attention scale, log-sum-exp statistics output, bottom-right causal mask,
 * additive bias, sink token).  The score matrix is computed tile by tile with
 * an online softmax (running max m and running sum l, rustytorch
 * flash_attention.metal, forward kernel) and never written to device memory.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Layout: q is [B, Hq, Lq, D], k and v are [B, Hkv, Lk, D], o is
 *    [B, Hq, Lq, D], element type params->dtype, dense row-major
 *    ("contiguous") unless SDPA_FLAG_STRIDES gives their strides (the D
 *    dimension stays contiguous).  lse is [B, Hq, Lq] float32, dense.  The query head h
 *    reads key/value head floor(h / (Hq / Hkv)) (contiguous head groups).
 *  - Pointers q, k, v, o, lse, mask, sinks and workspace are DEVICE pointers
 *    owned by the caller; the library never allocates, frees or retains them.
 *    Base pointers of q, k, v and o must be 16-byte aligned; mask aligned to
 *    its element size; lse, sinks 4-byte aligned; workspace 256-byte
 *    aligned.
 *  - sdpa_forward is asynchronous on `stream` (a cudaStream_t, passed as
 *    void* so that this header needs no CUDA include; NULL = legacy default
 *    stream).  It never synchronises the host.
 *  - Argument and layout errors are detected on the host before any launch,
 *    and nothing is written.  Launch failures are reported as SDPA_ERR_CUDA.
 *    No C++ exception crosses this ABI.  Kernels never trap: a device-side
 *    wait that gives up sets a device status word, read and cleared by
 *    sdpa_device_status().
 */
#ifndef GB300_SDPA_H_
#define GB300_SDPA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SDPA_ABI_VERSION 5

#if defined(__GNUC__)
#define SDPA_API __attribute__((visibility("default")))
#else
#define SDPA_API
#endif

typedef enum {
  SDPA_F32 = 0,
  SDPA_F16 = 1,
  SDPA_BF16 = 2
} sdpa_dtype_t;

typedef enum {
  SDPA_OK = 0,
  SDPA_ERR_INVALID_ARGUMENT = 1, /* null pointer, non-positive size, bad stride */
  SDPA_ERR_UNSUPPORTED = 2,      /* valid problem outside the supported space */
  SDPA_ERR_MISALIGNED = 3,       /* a base pointer breaks the alignment rule */
  SDPA_ERR_WORKSPACE_TOO_SMALL = 4,
  SDPA_ERR_CUDA = 5,             /* a CUDA runtime call or launch failed */
  SDPA_ERR_TIMEOUT = 6,          /* a device-side wait gave up (status word) */
  SDPA_ERR_PAGE_TABLE = 7,       /* a page number outside the cache was met
                                    (status word; paged entry points) */
  SDPA_ERR_POSITION = 8          /* a position outside the rotation table was
                                    met (status word; rotary entry points) */
} sdpa_status_t;

/* Kernel paths.  The launcher picks one from the shape alone: one query row
 * per head (decode), or a few (up to 2 at D = 64/128, up to 8 at D = 512),
 * take the split-KV vector path, where the rows of a kv head share its K/V
 * stream; longer query sequences take the prefill kernels. */
typedef enum {
  SDPA_KERNEL_NONE = 0,
  SDPA_KERNEL_PREFILL_TC = 1,   /* fp16/bf16, Lq > 2: TMA + tcgen05 + TMEM */
  SDPA_KERNEL_PREFILL_F32 = 2,  /* fp32, D = 128, Lq > 2: fp32 FMA tiles */
  SDPA_KERNEL_DECODE_SPLITKV = 3, /* small Lq: split-KV vector pass + merge */
  SDPA_KERNEL_NO_KEYS = 4,       /* Lk == 0: writes o = 0 and the empty lse */
  SDPA_KERNEL_PREFILL_TC_F32 = 5 /* fp32, D = 64, Lq > 2: bf16 hi/lo splits on
                                    tcgen05 (three products per step) */
} sdpa_kernel_t;

/*
 * Problem description.
 *  batch, num_q_heads, num_kv_heads, seq_len_q, seq_len_kv, head_dim:
 *      B, Hq, Hkv, Lq, Lk, D.  Hkv >= 1, the others >= 0, Hq % Hkv == 0,
 *      D in {64, 128, 512} (512: Lq <= 8 only), Lq and Lk at most 2^30.  When B * Hq * Lq == 0
 *      there is nothing to compute and the call returns SDPA_OK at once.
 *      When Lk == 0 every row sees no key: o = 0 and lse = -inf (the sink
 *      logit itself with sinks).
 *  dtype: element type of q, k, v, o and mask.
 *  scale: multiplies q.k before the mask is added; the caller passes it
 *      explicitly (1/sqrt(D) for the usual choice).  Must be finite.
 *  causal: nonzero = bottom-right aligned causal mask, key j is visible to
 *      query i iff j <= i + (Lk - Lq) (the alignment of the cuDNN graph's
 *      causal_mask_bottom_right; identical to "j <= i" when Lq == Lk).
 *      Requires Lq <= Lk.
 *  mask: NULL or an additive bias added to the scaled scores, element type
 *      dtype, addressed as mask[b*s0 + h*s1 + i*s2 + j*s3] with
 *      mask_stride = {s0, s1, s2, s3} in ELEMENTS; a stride of 0 broadcasts
 *      that dimension; s3 must be 1.  -inf entries remove a key.  With
 *      SDPA_FLAG_BOOL_MASK it is a boolean mask instead: one byte per
 *      element (same addressing, strides in bytes), nonzero = the key is
 *      visible to the query, zero = removed.  When both mask and causal are
 *      given, both apply.
 *  sinks: NULL or float32 [Hq]: one extra logit per query head that enters
 *      the softmax denominator only (a key with a zero value row).  It is
 *      not multiplied by scale and not masked.
 *  kv_capacity: 0, or the number of rows per (batch, kv head) that k and v
 *      hold (>= seq_len_kv): k and v are then [B, Hkv, kv_capacity, D], a
 *      fixed-capacity KV cache of which rows [0, seq_len_kv) are used (the
 *      rest is never read into a result).  0 means kv_capacity = seq_len_kv.
 *  seq_lens_q, seq_lens_kv: NULL, or DEVICE int32 [B] arrays of per-batch
 *      lengths (padding masks): batch b uses query rows [0, seq_lens_q[b])
 *      and keys [0, seq_lens_kv[b]) (values are clamped to [0, seq_len_q]
 *      and [0, seq_len_kv]); query rows at or past its length see no key
 *      (o = 0, lse = -inf or the sink), and the bottom-right causal rule
 *      uses the batch's own lengths: key j visible to query i iff
 *      j <= i + (seq_lens_kv[b] - seq_lens_q[b]).  Both arrays must stay
 *      valid until the call's kernels have run.  The prefill kernels and
 *      the fp16/bf16 decode passes load whole key
 *      tiles, so v rows [seq_lens_kv[b], seq_len_kv) meet zero weights there
 *      and must hold finite values (rows past seq_len_kv are never read).
 *  flags: an OR of the SDPA_FLAG_* bits below (other bits must be 0, else
 *      SDPA_ERR_INVALID_ARGUMENT).
 *  q_stride, k_stride, v_stride, o_stride (ABI 4): read only with
 *      SDPA_FLAG_STRIDES (a caller built against ABI 3 leaves the flag clear
 *      and need not provide them).  Element strides of dimensions B, H and L
 *      of each tensor (D is contiguous), each >= 0 and, times the element
 *      size, a multiple of 16 bytes; o must not overlap q, k or v.  They
 *      replace the dense layout and kv_capacity (which must then be 0).
 *      Example: [B, L, H, D] tensors ("BSHD") have strides {L*H*D, D, H*D}.
 */
/* The call runs beside other work on the GPU (kernels of other streams):
 * launch shapes are not fitted to an idle GPU.  Without it, a prefill whose
 * query-tile units leave a partial last wave on the SMs shares the key tiles
 * of those units among the CTAs of thread-block clusters (a second, shorter
 * grid); with it, every unit runs whole. */
#define SDPA_FLAG_SHARED_GPU 0x1u
/* mask is boolean (bytes, nonzero = visible) instead of an additive bias. */
#define SDPA_FLAG_BOOL_MASK 0x2u
/* q_stride, k_stride, v_stride and o_stride give the tensors' layouts. */
#define SDPA_FLAG_STRIDES 0x4u
typedef struct {
  int32_t batch;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t seq_len_q;
  int32_t seq_len_kv;
  int32_t head_dim;
  int32_t dtype;   /* sdpa_dtype_t */
  float scale;
  int32_t causal;
  int32_t reserved0;
  const void* mask;
  int64_t mask_stride[4];
  const float* sinks;
  int32_t kv_capacity;          /* ABI 2 */
  uint32_t flags;               /* ABI 3 (was reserved, 0) */
  const int32_t* seq_lens_q;    /* ABI 2 */
  const int32_t* seq_lens_kv;   /* ABI 2 */
  int64_t q_stride[3];          /* ABI 4, with SDPA_FLAG_STRIDES */
  int64_t k_stride[3];
  int64_t v_stride[3];
  int64_t o_stride[3];
} sdpa_params_t;

/*
 * sdpa_workspace_size — bytes of device workspace that sdpa_forward needs for
 * this problem (split-KV partial outputs of the decode path; the bf16 hi/lo
 * copies of q, k and v of the fp32 tensor-core prefill; for an fp16/bf16
 * prefill whose mask has a row per query, room for a copy of the mask laid
 * out in the kernel's 128 x 128 score tiles — optional: with a smaller or
 * NULL workspace that call reads the mask where it lies, slower where a
 * warp's rows are far apart; 0 when the chosen path needs none).  Pure host
 * function; returns 0 for an invalid problem as well (sdpa_forward then
 * reports the error).
 */
SDPA_API size_t sdpa_workspace_size(const sdpa_params_t* params);

/*
 * sdpa_select_kernel — the kernel path sdpa_forward would run for this
 * problem, or SDPA_KERNEL_NONE with *status set when the problem is invalid
 * or unsupported (SDPA_KERNEL_NONE with SDPA_OK: nothing to compute).  Pure
 * host function (no CUDA call).  `status` may be NULL.
 */
SDPA_API sdpa_kernel_t sdpa_select_kernel(const sdpa_params_t* params, sdpa_status_t* status);

/*
 * sdpa_forward — compute o (and lse, when non-NULL) for the problem in
 * `params` on `stream`.
 *  q, k, v: inputs (device, read only).  o: output (device, written).
 *  lse: NULL or float32 [B, Hq, Lq] output in natural-log units; a fully
 *      masked row gives o = 0 and lse = -inf (lse = sink with sinks).
 *  workspace / workspace_bytes: device scratch of at least
 *      sdpa_workspace_size(params) bytes (NULL allowed when that is 0).  Its
 *      contents need no initialisation and are overwritten; two calls that
 *      overlap on the GPU must not share one workspace.
 * Returns SDPA_OK once the work is enqueued.
 */
SDPA_API sdpa_status_t sdpa_forward(const sdpa_params_t* params,
                           const void* q, const void* k, const void* v,
                           void* o, float* lse,
                           void* workspace, size_t workspace_bytes,
                           void* stream);

/*
 * sdpa_backward_workspace_size — bytes of device workspace that sdpa_backward
 * needs (an fp32 dQ accumulator [B, Hq, Lq, D] and two fp32 [B, Hq, Lq]
 * arrays); 0 for an invalid or unsupported problem.  Pure host function.
 */
SDPA_API size_t sdpa_backward_workspace_size(const sdpa_params_t* params);

/*
 * sdpa_backward — gradients of the forward pass (the backward kernels of the
 * rustytorch flash_attention.metal page: P = exp(S - LSE), D_i = dO_i . O_i,
 * dS = P (dO V^T - D), dQ = scale dS K, dK = scale dS^T Q, dV = P^T dO; with
 * the options of the mlx cuDNN backward graph: scale, bottom-right causal
 * mask, additive or boolean mask, sink token).  The problem description is
 * the forward's (same params), per-batch length arrays included: rows and
 * keys past a batch's lengths get zero gradients.  Supported: head_dim 64 or
 * 128 (else SDPA_ERR_UNSUPPORTED); fp16/bf16 on the tensor cores, fp32 on
 * fp32 CUDA-core kernels.  Rows of q, k, v and d_o inside seq_len_q /
 * seq_len_kv but past a batch's lengths must hold finite values (whole tiles
 * are read; their weights are zero).
 *  q, k, v, o, lse: the forward's inputs, output and log-sum-exp (lse is
 *      required: the forward must have been asked for it).
 *  d_o: gradient of the loss with respect to o, in o's layout.
 *  dq, dk, dv: outputs in the layouts of q, k and v (their dtype).  With
 *      grouped-query heads dk and dv sum over the query heads of each group.
 *      The sink and the mask receive no gradient.
 *  workspace / workspace_bytes: at least sdpa_backward_workspace_size(params)
 *      bytes, 256-byte aligned; contents need no initialisation.
 * Asynchronous on `stream`; errors as for sdpa_forward.
 */
SDPA_API sdpa_status_t sdpa_backward(const sdpa_params_t* params, const void* q, const void* k,
                                     const void* v, const void* o, const void* d_o,
                                     const float* lse, void* dq, void* dk, void* dv,
                                     void* workspace, size_t workspace_bytes, void* stream);

/*
 * sdpa_host_staging_size — bytes of device staging memory that
 * sdpa_forward_host needs for this problem cut into `pieces` pieces (device
 * copies of q, k, v, o and lse, and two workspaces); 0 for a problem that
 * sdpa_forward_host rejects.  Pure host function.
 */
SDPA_API size_t sdpa_host_staging_size(const sdpa_params_t* params, int pieces);

/*
 * sdpa_forward_host — sdpa_forward for callers whose q, k, v and results
 * live in host memory: the whole trip of the mlx page's call (mlx 0.30.7
 * scaled_dot_product_attention.cpp, eval_gpu: the framework's arrays brought
 * to the device, the fused graph run, the output handed back), with the
 * transfers of one piece overlapping the kernels of another.
 *  q_host, k_host, v_host: inputs in HOST memory, dense [B, H, L, D] in
 *      params->dtype (page-locked memory, cudaMallocHost or
 *      cudaHostRegister, lets the copies overlap; pageable memory works, with
 *      each copy waiting for the host).
 *  o_host, lse_host: outputs in host memory, dense (lse_host may be NULL).
 *  params: as for sdpa_forward; mask and sinks, if any, are DEVICE pointers.
 *      Dense layouts only: SDPA_FLAG_STRIDES, a kv_capacity other than 0 or
 *      seq_len_kv, or per-batch length arrays give SDPA_ERR_UNSUPPORTED.
 *  staging / staging_bytes: caller-owned device memory of at least
 *      sdpa_host_staging_size(params, pieces) bytes, 256-byte aligned; two
 *      calls whose work overlaps must not share it.
 *  pieces: the (batch, kv-head) pairs are cut into about this many pieces,
 *      each within one batch.  Piece i's host-to-device copies run on two
 *      copy streams, its kernels (those of sdpa_forward, with
 *      SDPA_FLAG_SHARED_GPU) on one of two compute streams, its
 *      device-to-host copies on a fifth: one cudaMemcpyAsync per piece and
 *      tensor.
 *  stream: the caller's stream.  The work starts after what is already
 *      enqueued on it, and what the caller enqueues on it afterwards runs
 *      after this call's copies have landed in o_host and lse_host (e.g. a
 *      cudaStreamSynchronize(stream) makes them readable).
 * The five streams and their events belong to the library: created on the
 * first call on a device (with that device current) and kept until exit;
 * calls from several threads are serialised while they enqueue.  Nothing is
 * allocated on the device.  sdpa_last_launch_count counts the kernels of
 * every piece.  Errors as for sdpa_forward; SDPA_ERR_WORKSPACE_TOO_SMALL for
 * too small a staging area.
 */
SDPA_API sdpa_status_t sdpa_forward_host(const sdpa_params_t* params, const void* q_host,
                                         const void* k_host, const void* v_host, void* o_host,
                                         float* lse_host, void* staging, size_t staging_bytes,
                                         int pieces, void* stream);

/* sdpa_status_string — static, NUL-terminated text for a status code. */
SDPA_API const char* sdpa_status_string(sdpa_status_t status);

/*
 * sdpa_device_status — synchronise `stream`, then read and clear the device
 * status word that kernels set when one of their bounded waits gives up, a
 * page table names a page outside the cache or a token's position lies outside
 * the rotation table.  Returns SDPA_OK, SDPA_ERR_TIMEOUT, SDPA_ERR_PAGE_TABLE,
 * SDPA_ERR_POSITION (the last one met), or SDPA_ERR_CUDA if the
 * synchronisation itself failed.  The status word is per device and shared by all streams.
 */
SDPA_API sdpa_status_t sdpa_device_status(void* stream);

/*
 * sdpa_debug_set_wait_limit_ns — test hook: upper bound in nanoseconds on
 * every device-side barrier wait of later launches (default 2e9).  0
 * restores the default.  Returns the previous value.
 */
SDPA_API uint64_t sdpa_debug_set_wait_limit_ns(uint64_t ns);

/*
 * sdpa_debug_set_option — test hooks that override a launch decision of
 * later calls, process-wide (they exist so that tests reach paths that the
 * planner would not pick for the test's sizes).  Returns the previous value;
 * an unknown option returns -1 and changes nothing.
 *  SDPA_DEBUG_DECODE_SPLITS   split count of the decode passes (0: the plan's)
 *  SDPA_DEBUG_DECODE_CLUSTER  0: never merge the splits inside a cluster
 *                             (two passes); 1: as planned (default)
 *  SDPA_DEBUG_DECODE_DROP_LAST 1: the vector path's producer skips its last
 *                             copy, so that a bounded wait runs out and the
 *                             call reports SDPA_ERR_TIMEOUT (default 0)
 *  SDPA_DEBUG_PREFILL_SPLIT   -1: the plan's (default); 0: never split the
 *                             last wave; 2, 4: every unit shared by that
 *                             many CTAs of a cluster
 *  SDPA_DEBUG_DECODE_VECTOR   1: head_dim-64/128 fp16/bf16 decode on the
 *                             vector path instead of the tensor-core pass
 *                             (default 0)
 *  SDPA_DEBUG_PAGED_SIMT      1: sdpa_paged_forward and sdpa_paged_scores of
 *                             every type on the CUDA-core tile kernels
 *                             (default 0)
 *  SDPA_DEBUG_PAGED_CTAS      CTAs that share the work of sdpa_paged_forward
 *                             and sdpa_paged_scores (0: the plan's; at most
 *                             the plan's)
 */
typedef enum {
  SDPA_DEBUG_DECODE_SPLITS = 0,
  SDPA_DEBUG_DECODE_CLUSTER = 1,
  SDPA_DEBUG_DECODE_DROP_LAST = 2,
  SDPA_DEBUG_PREFILL_SPLIT = 3,
  SDPA_DEBUG_DECODE_VECTOR = 4,
  SDPA_DEBUG_PAGED_SIMT = 5,
  SDPA_DEBUG_PAGED_CTAS = 6
} sdpa_debug_option_t;
SDPA_API int sdpa_debug_set_option(int option, int value);

/* sdpa_abi_version — SDPA_ABI_VERSION of the built library. */
SDPA_API int sdpa_abi_version(void);

/*
 * sdpa_last_launch_count — number of kernels that the calling thread's last
 * sdpa_forward or sdpa_forward_decode_noalloc call enqueued (0 if it
 * returned an error or had nothing to compute): 1 for the prefill kernels
 * and for a decode whose splits merge inside a thread-block cluster, 2 for
 * the fp32 hi/lo prefill (split, then prefill) and the two-pass decode.
 * Host function, no CUDA call.
 */
SDPA_API int sdpa_last_launch_count(void);

/*
 * sdpa_forward_decode_noalloc — the vector path (decode) without a
 * caller workspace.  The pages have no counterpart: this entry point exists
 * for callers that cannot call cudaMalloc or pass device scratch where they
 * run attention (a stream being captured into a CUDA graph may not
 * allocate, cudaMalloc can synchronise the device, and some hosts own every
 * device byte through their own pool and have none to spare for a library).
 *
 * Same problem description, inputs, outputs, stream and errors as
 * sdpa_forward, restricted to problems that sdpa_select_kernel maps to
 * SDPA_KERNEL_DECODE_SPLITKV (others: SDPA_ERR_UNSUPPORTED; nothing to
 * compute: SDPA_OK).  The split-KV partial results go to one static device
 * array of SDPA_NOALLOC_SCRATCH_BYTES (8 MiB) that every GPU loading the
 * library holds until exit; a problem whose partial results do not fit
 * (about B * Hq * Lq * splits * (D + 1) * 4 bytes) returns
 * SDPA_ERR_WORKSPACE_TOO_SMALL before any launch.  Nothing is allocated.
 *  - The first call on a device (with that device current) looks up the
 *    array's device address (cudaGetSymbolAddress) and caches it: make that
 *    first call before any stream capture.
 *  - All calls on a device share the array and it keeps the last call's
 *    contents; calls whose kernels overlap on the GPU race on it, so the
 *    caller must order them (one stream, or events).  Nothing in it needs to
 *    start at zero: each call writes every partial result before reading it.
 */
#define SDPA_NOALLOC_SCRATCH_BYTES (8u * 1024u * 1024u)
SDPA_API sdpa_status_t sdpa_forward_decode_noalloc(const sdpa_params_t* params,
                                                   const void* q, const void* k,
                                                   const void* v, void* o, float* lse,
                                                   void* stream);

/* ------------------------------------------------------- paged KV cache ---
 * Keys and values of many sequences in pages of a shared pool, as a serving
 * loop keeps them: each step writes the new tokens' K and V rows
 * (sdpa_paged_write), attends from the new tokens over everything cached
 * (sdpa_paged_forward), may add up the attention weight that each cached key
 * received (sdpa_paged_scores) and, when a sequence outgrows its budget,
 * drops the keys of least accumulated weight (sdpa_paged_evict).
 *
 * Conventions shared by the four calls
 *  - The cache: k_pages and v_pages are [num_pages, Hkv, page_size, D] by
 *    shape with element strides k_stride / v_stride = {page, head, row} (D
 *    contiguous), so that both storage orders, rows before heads
 *    ([page][row][head][D]) and heads before rows, are served.  Position p of
 *    sequence b is row p % page_size of page
 *    page_table[b * page_table_stride + p / page_size] (device int32, at
 *    most max_pages entries a sequence).  Entries that no position below the
 *    sequence's length uses are not read.  An entry outside [0, num_pages)
 *    reads as zero keys and values (written rows are dropped) and sets the
 *    device status word to SDPA_ERR_PAGE_TABLE.
 *  - seq_lens_kv: device int32 [num_seqs], the keys of each sequence with its
 *    new tokens included (negative: 0).  Positions at or past max_pages *
 *    page_size have no place in the cache: nothing is written there, no token
 *    sees them, and sdpa_paged_evict counts the keys before them only.  The new
 *    tokens of such a length keep their positions; those past the end see every
 *    key that has a place.
 *  - New tokens are packed: q is [num_tokens, Hq, D] with element strides
 *    q_stride = {token, head}; the tokens of sequence b are rows
 *    [cu_seqlens_q[b], cu_seqlens_q[b + 1]) (device int32 [num_seqs + 1],
 *    non-decreasing, clamped to [0, num_tokens]).  cu_seqlens_q NULL: one
 *    token a sequence, row b.  They are the sequence's last positions: token
 *    i of nq sits at position nk - nq + i, nk the length.  Rows past the last
 *    sequence's end belong to none: their rows of o and lse are left as they
 *    were.
 *  - causal nonzero (the usual case): a token sees the keys at and before
 *    its own position; zero: every key of its sequence.  A token that sees
 *    no key (nq > nk) gives o = 0 and lse = -inf, or the sink.
 *  - The cache's rows below a sequence's length hold finite values (a row
 *    meets the weight 0 of tokens that do not see it); rows at or past it may
 *    hold anything, NaN included.  The lengths, offsets and page tables do not
 *    change while a call runs.
 *  - head_dim 64 or 128; fp32, fp16, bf16; any Hq that Hkv divides; page_size
 *    >= 1.  fp16/bf16 with page_size a multiple of 8 and a positive scale run
 *    on the tensor cores, everything else on fp32 CUDA-core kernels.  Scores,
 *    sums and outputs are held in fp32 and o is rounded once.  On the tensor
 *    cores sdpa_paged_forward also rounds each softmax weight to the cache's
 *    type before it meets its value row (2^-8 relative in bf16, 2^-11 in fp16;
 *    lse and the accumulated weights are not affected).
 *  - Base pointers 16-byte aligned, row strides multiples of 16 bytes; o must
 *    not overlap the inputs.  sdpa_paged_write and sdpa_paged_evict want k_pages
 *    and v_pages without a common row (interleaved is fine; one cache for both
 *    is refused, unless the rows written are the same too).  flags and reserved
 *    fields must be 0.
 *  - Asynchronous on `stream`, nothing allocated, results independent of
 *    timing (fixed summation order).  Host-side errors as for sdpa_forward.
 *    Two calls that overlap on the GPU must not share a workspace.
 */
typedef struct {
  int32_t num_seqs;
  int32_t num_tokens;    /* rows of q (and of the new k and v) */
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t dtype;         /* sdpa_dtype_t of q, o and the cache */
  float scale;
  int32_t causal;
  int32_t num_pages;
  int32_t page_size;
  int32_t max_pages;
  uint32_t flags;        /* 0 */
  const int32_t* page_table;
  int64_t page_table_stride;   /* elements between sequences */
  const int32_t* cu_seqlens_q; /* or NULL */
  const int32_t* seq_lens_kv;
  const float* sinks;          /* NULL or float32 [Hq] (sdpa_paged_forward) */
  int64_t q_stride[2];
  int64_t o_stride[2];
  int64_t k_stride[3];
  int64_t v_stride[3];
} sdpa_paged_params_t;

/*
 * sdpa_paged_write — copy the new tokens' key and value rows into the cache.
 *  k, v: [num_tokens, Hkv, D] with element strides k_new_stride and
 *      v_new_stride = {token, head}.  Token i of sequence b goes to position
 *      nk - nq + i; a token whose position is negative or past max_pages *
 *      page_size is not written.  num_q_heads, scale, causal, sinks, q_stride
 *      and o_stride are not used.
 */
SDPA_API sdpa_status_t sdpa_paged_write(const sdpa_paged_params_t* params, const void* k,
                                        const void* v, const int64_t* k_new_stride,
                                        const int64_t* v_new_stride, void* k_pages,
                                        void* v_pages, void* stream);

/*
 * sdpa_paged_workspace_size — bytes of device workspace that
 * sdpa_paged_forward and sdpa_paged_scores need for this problem (partial
 * results of work that is shared among CTAs; a function of head_dim and the
 * device's SM count alone: 40 MB at head_dim 128 on 152 SMs); 0 for an invalid
 * problem or one with nothing to compute.
 */
SDPA_API size_t sdpa_paged_workspace_size(const sdpa_paged_params_t* params);

/*
 * sdpa_paged_forward — attention of the new tokens over the paged cache.
 *  q: [num_tokens, Hq, D]; o: the same shape, strides o_stride.
 *  lse: NULL or float32 [num_tokens, Hq], dense, natural-log units.
 *  workspace: at least sdpa_paged_workspace_size(params) bytes, 256-byte
 *      aligned; contents need no initialisation.
 */
SDPA_API sdpa_status_t sdpa_paged_forward(const sdpa_paged_params_t* params, const void* q,
                                          const void* k_pages, const void* v_pages, void* o,
                                          float* lse, void* workspace, size_t workspace_bytes,
                                          void* stream);

/*
 * sdpa_paged_scores — add the attention weight that every cached key receives
 * from the new tokens:
 *     scores[b, kvh, j] += sum over the tokens i of sequence b that see key j
 *                          and the query heads h of kvh of
 *                          exp(scale * q_i,h . k_j - lse_i,h)
 *  lse: float32 [num_tokens, Hq] as sdpa_paged_forward left it (with sinks,
 *      if any, in it).  scores: float32, element (b, kvh, j) at b *
 *      score_stride[0] + kvh * score_stride[1] + j for j < score_len; keys at
 *      or past score_len and scores at or past a sequence's length are left
 *      alone.  A row whose lse is -inf adds nothing.  v_stride, o_stride and
 *      sinks are not used.
 */
SDPA_API sdpa_status_t sdpa_paged_scores(const sdpa_paged_params_t* params, const void* q,
                                         const void* k_pages, const float* lse, float* scores,
                                         const int64_t* score_stride, int32_t score_len,
                                         void* workspace, size_t workspace_bytes, void* stream);

/*
 * sdpa_paged_evict — cut every sequence longer than `keep` (>= 1) back to
 * `keep` keys per kv head: its newest min(recent, keep) keys stay, and of the
 * others those of largest score (ties to the lower position; NaN counts as
 * -inf, 0 and -0 tie).  The kept rows of K and V move, in order, to positions
 * 0, 1, ... of the sequence's own pages; the heads choose independently.
 * Sequences of at most `keep` keys stay as they are.  keep and score_len are
 * at most 2^30.
 *  scores: float32 [num_seqs, Hkv, score_len] as for sdpa_paged_scores; keys
 *      at or past score_len count as score 0.
 *  scores_out: NULL or the kept keys' scores in their new places, 0 behind
 *      them up to score_len; may be `scores` itself.
 *  kept: int32 [num_seqs, Hkv, keep], dense: the old positions, ascending, -1
 *      behind the last.
 *  seq_lens_out: NULL or int32 [num_seqs], min(length, keep); may be
 *      params->seq_lens_kv itself.
 * A kept row of a page outside the cache arrives as zeros, and one that would
 * move to such a page is dropped (SDPA_ERR_PAGE_TABLE in the status word).
 * The pages that a sequence longer than `keep` uses below position `keep`
 * are rewritten, so no other sequence may share them, and no page may appear
 * twice among a sequence's own.  num_tokens, num_q_heads, scale, causal,
 * cu_seqlens_q, sinks, q_stride and o_stride are not used.
 */
SDPA_API sdpa_status_t sdpa_paged_evict(const sdpa_paged_params_t* params, int32_t keep,
                                        int32_t recent, void* k_pages, void* v_pages,
                                        const float* scores, float* scores_out,
                                        const int64_t* score_stride, int32_t score_len,
                                        int32_t* kept, int32_t* seq_lens_out, void* stream);

/* ------------------------------------------------------ rotary positions ---
 * Pair i of a head, i < R / 2, turns by the angle of its token's position:
 *     (x, y) -> (x cos - y sin, y cos + x sin)
 * with the pairs (i, i + R / 2), or (2 i, 2 i + 1) where `interleaved`; the
 * elements from R on pass unchanged.  The rotation is computed in fp32 and
 * rounded once.
 */
typedef struct {
  const float* table;       /* [table_len, rotary_dim / 2, 2]: cosine and sine
                               of every position and pair, 16-byte aligned */
  int64_t table_len;
  int32_t rotary_dim;       /* R: a multiple of 16, at most head_dim */
  int32_t interleaved;
  const int32_t* positions; /* device int32, or NULL: see the calls */
} sdpa_rotation_t;

/*
 * sdpa_rope_table — fill a rotation table: entry (p, i) is (gain * cos, gain *
 * sin) of p * inv_freq[i], the angle and its functions in 64 bits, rounded
 * once.  table: device float32 [length, rotary_dim / 2, 2], 16-byte aligned.
 * inv_freq: HOST array of rotary_dim / 2 numbers (rotary_dim a multiple of 16,
 * at most 512), read before the call returns.
 */
SDPA_API sdpa_status_t sdpa_rope_table(float* table, int64_t length, int32_t rotary_dim,
                                       const double* inv_freq, double gain, void* stream);

/*
 * sdpa_rope — rotate q and k.  q: [B, Hq, L, D], k: [B, Hkv, L, D], D 64, 128
 * or 512, element strides {batch, head, row} (D contiguous; times the element
 * size multiples of 16 bytes); q_out and k_out likewise, either the input
 * itself (same pointer and strides) or without a common element with the
 * inputs and each other.  num_kv_heads 0 (k and k_out unused) rotates q alone.
 * rotation.positions: int32, token (b, l) at b * position_stride + l (a stride
 * of 0 shares them among the batches); NULL: l itself.  A position outside
 * [0, table_len) leaves its row as it is and sets the device status word to
 * SDPA_ERR_POSITION.
 * transpose nonzero: the transposed rotation, which takes the gradients of
 * q_out and k_out to those of q and k (with a table of gain 1 the inverse).
 */
typedef struct {
  int32_t batch;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t seq_len;
  int32_t head_dim;
  int32_t dtype;      /* sdpa_dtype_t of all four tensors */
  int32_t transpose;
  uint32_t flags;     /* 0 */
  sdpa_rotation_t rotation;
  int64_t position_stride;
  int64_t q_stride[3];
  int64_t k_stride[3];
  int64_t q_out_stride[3];
  int64_t k_out_stride[3];
} sdpa_rope_params_t;
SDPA_API sdpa_status_t sdpa_rope(const sdpa_rope_params_t* params, const void* q, const void* k,
                                 void* q_out, void* k_out, void* stream);

/*
 * sdpa_paged_append — rotate a step's new tokens and write them to the paged
 * cache: sdpa_rope and sdpa_paged_write in one pass.
 *  q, q_out: [num_tokens, Hq, D], strides params->q_stride and o_stride; q_out
 *      is q itself (same strides) or has no common element with the inputs.
 *      num_q_heads 0: no queries (q and q_out unused).
 *  k, v, k_new_stride, v_new_stride, k_pages, v_pages: as for
 *      sdpa_paged_write; k is rotated, rounded to its type and written, v
 *      written as it is.
 *  rotation->positions: int32 [num_tokens], or NULL: token i of the nq of
 *      sequence b is at position seq_lens_kv[b] - nq + i.  A token whose
 *      position the table does not hold keeps its q and k unrotated and sets
 *      the status word to SDPA_ERR_POSITION (but not one before the sequence's
 *      start, which has no place in the cache either).
 * Rows of q_out of tokens that belong to no sequence are left as they were.
 * scale, causal and sinks are not used.
 */
SDPA_API sdpa_status_t sdpa_paged_append(const sdpa_paged_params_t* params,
                                         const sdpa_rotation_t* rotation, const void* q,
                                         const void* k, const void* v, void* q_out,
                                         const int64_t* k_new_stride,
                                         const int64_t* v_new_stride, void* k_pages,
                                         void* v_pages, void* stream);

/* --------------------------------------------------- 4-bit paged KV cache ---
 * The paged cache at 4.5 bits an element.  A row of D elements is D / 2 bytes of
 * codes, two 4-bit floats each (sign, 2 exponent bits, 1 mantissa bit: 0, 0.5,
 * 1, 1.5, 2, 3, 4, 6), the even element in the low half, and D / 16 scales, an
 * 8-bit float (4 exponent bits, 3 mantissa bits; e4m3) for 16 consecutive
 * elements.  An element stands for code * scale * g, g its kv head's gain.
 * A row x in its own type is written as follows: y = x / g in fp32; the scale
 * is max |y| over the 16 elements, divided by 6 and rounded to e4m3, at least
 * 2^-9 and at most 448; the code is y / scale rounded to the nearest code, ties
 * to even, at most 6 in magnitude (zeros are stored as code 0).  Rows hold
 * finite values (an infinity is stored as the largest value, a NaN as some
 * finite one).
 *
 * Codes and scales are two tensors of bytes for K and two for V, [num_pages,
 * Hkv, page_size, D / 2] and [num_pages, Hkv, page_size, D / 16] by shape; the
 * codes' byte strides {page, head, row} are k_stride and v_stride of
 * sdpa_paged_params_t (multiples of 16), the scales' are here (multiples of
 * D / 16).  Codes 16-byte aligned, scales D / 16 bytes.  Everything else is as
 * for the paged cache above: page tables, lengths, packed tokens, status word.
 */
typedef struct {
  void* k_codes;
  void* v_codes;
  void* k_scales;
  void* v_scales;
  int64_t k_scale_stride[3];
  int64_t v_scale_stride[3];
  const float* k_gain; /* NULL (1), or device float32 [Hkv] of magnitudes
                          between 2^-100 and 2^100 */
  const float* v_gain;
} sdpa_fp4_cache_t;

/*
 * sdpa_paged_append_fp4 — sdpa_paged_append into a 4-bit cache.
 *  rotation: NULL leaves q and k unrotated (num_q_heads 0 then, or q is
 *      copied).
 *  k_out, v_out: NULL, or [num_tokens, Hkv, D] in params->dtype with strides
 *      out_stride = {token, head}: what the written rows stand for, rounded to
 *      the type (the same for a token without a place in the cache; rows of
 *      tokens of no sequence are left as they were).  They overlap no other
 *      tensor of the call.
 */
SDPA_API sdpa_status_t sdpa_paged_append_fp4(const sdpa_paged_params_t* params,
                                             const sdpa_rotation_t* rotation,
                                             const sdpa_fp4_cache_t* cache, const void* q,
                                             const void* k, const void* v, void* q_out,
                                             const int64_t* k_new_stride,
                                             const int64_t* v_new_stride, void* k_out,
                                             void* v_out, const int64_t* out_stride,
                                             void* stream);

/*
 * sdpa_paged_forward_fp4 — sdpa_paged_forward over a 4-bit cache.  q, o and
 * lse as there, in params->dtype; workspace of sdpa_paged_workspace_size bytes.
 * A scale byte of NaN below a sequence's length gives NaN.
 * Rounding: scores, sums and lse are fp32.  bf16 queries lose what is below 2^-39
 * of their row's largest element; fp32 ones are held to 2^-22 of an element, or
 * 2^-39 of that.  A softmax weight meets its value as an fp16 number (2^-11 of it,
 * or 2^-29 of the row's largest weight, whichever is more), in fp32 calls as two
 * (2^-22, or 2^-41).  o is rounded once.
 */
SDPA_API sdpa_status_t sdpa_paged_forward_fp4(const sdpa_paged_params_t* params,
                                              const sdpa_fp4_cache_t* cache, const void* q,
                                              void* o, float* lse, void* workspace,
                                              size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GB300_SDPA_H_ */
