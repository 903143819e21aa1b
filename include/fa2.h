/*
 * fa2.h -- C ABI of the GB300 (sm_103a) exact tiled attention: forward pass,
 * its backward pass and a decoding-regime forward.
 *
 * The operation (FlashAttention V2 in depth, section 6.1 "Full forward
 * algorithm"; Flash Attention 2 page, "Standard Attention" and "Causal
 * masking"): for every batch b and head h, with S = scale * Q K^T and, when
 * causal, S_ij = -inf for key j > query i,
 *
 *     O   = softmax_row(S) V                      (exact, not approximate)
 *     LSE = m + ln(l),  m = rowmax(S),  l = rowsum(exp(S - m))
 *
 * computed in query tiles that stream key/value tiles through on-chip memory
 * with an online softmax, so the N x N score matrix never reaches global
 * memory.  LSE is the natural-log logsumexp that section 7.1 keeps for the
 * backward pass.
 *
 * Entry points:
 *   fa2_fwd / fa2_bwd        contiguous [B, H, N, d] tensors (fp16 or bf16),
 *                            lse [B, H, N] float32, full or causal attention;
 *   fa2_fwd_ex / fa2_bwd_ex  any strides, N_q != N_k, band and prefix masks,
 *                            packed variable-length batches (fa2_fwd_params);
 *   fa2_decode               up to FA2_DECODE_MAX_Q query rows per sequence
 *                            against long key sequences (fa2_fwd_params);
 *   fa2_fwd_host[_noalloc]   the forward on host buffers, end to end;
 *   fa2_paged_plan / fa2_paged_append / fa2_paged_fwd
 *                            a serving step on a paged key/value cache: block
 *                            tables and slots from request lengths, new rows
 *                            written to their slots, attention of each
 *                            request's new tokens (grouped query heads).
 *
 * Ownership: the caller owns every buffer.  fa2_fwd and fa2_fwd_ex allocate
 * no device memory; fa2_bwd, fa2_bwd_ex, fa2_decode and fa2_paged_fwd take a
 * caller workspace.  The library keeps one small device status word per device
 * for reporting kernel-side wait timeouts, rejected packed offsets and
 * out-of-range pages (see fa2_get_device_status).
 *
 * No C++ exception crosses this interface: every entry point returns an
 * fa2_status code.
 */
#ifndef FA2_GB300_H
#define FA2_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of q, k, v and o. */
typedef enum { FA2_FP16 = 0, FA2_BF16 = 1 } fa2_dtype;

typedef enum {
  FA2_OK = 0,
  FA2_ERR_INVALID_ARG = 1,    /* bad size, dtype, scale, null pointer or aliasing */
  FA2_ERR_UNSUPPORTED = 2,    /* head dim not in {64, 128, 256}, or no sm_103 device */
  FA2_ERR_MISALIGNED = 3,     /* a pointer is not 16-byte aligned */
  FA2_ERR_CUDA = 4,           /* a CUDA runtime/driver call failed */
  FA2_ERR_DEVICE_TIMEOUT = 5, /* a kernel wait ran out of time (fa2_get_device_status) */
  FA2_ERR_SCRATCH_LIMIT = 6,  /* problem too large for fa2_fwd_host_noalloc's static scratch */
  FA2_ERR_DEVICE_SEQLENS = 7, /* packed-batch offsets out of range (fa2_get_device_status) */
  FA2_ERR_DEVICE_PAGES = 8    /* paged cache: lengths, slots or pages out of range (fa2_get_device_status) */
} fa2_status;

/*
 * fa2_fwd -- forward pass on device buffers (asynchronous on `stream`).
 *
 *   q, k, v : device pointers, [B, H, N, d] `dtype`, read only, 16-byte aligned
 *   o       : device pointer, [B, H, N, d] `dtype`, written (RN-even from fp32)
 *   lse     : device pointer, [B, H, N] float32, written (natural log)
 *   B, H, N : batch, heads, sequence length (each >= 1; B*H*N*d < 2^31 elements
 *             per tensor is not required, but B*H < 2^31 and N < 2^31 are)
 *   d       : head dimension, one of 64, 128, 256 (the pages cap head dim at 256)
 *   scale   : any finite value (0: uniform weights over the visible keys; a
 *             negative scale reverses the score order); the pages use 1/sqrt(d)
 *   causal  : 0 = every key visible; 1 = key j visible to query i iff j <= i
 *   dtype   : FA2_FP16 or FA2_BF16
 *   stream  : a cudaStream_t (0 = legacy default stream)
 *
 * Every argument is checked before any CUDA call; a bad argument returns its
 * code and launches nothing.  o and lse must not overlap q, k or v.  The call
 * does not synchronise; kernel-side failures surface through
 * fa2_get_device_status.  The result is deterministic (no atomics; every
 * output element is written once).
 */
int fa2_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
            int B, int H, int N, int d, float scale, int causal, int dtype, void* stream);

/*
 * fa2_fwd_params -- arguments of fa2_fwd_ex, the general forward pass:
 * strided layouts, unequal query and key lengths, band and prefix masks and
 * packed variable-length batches.
 *
 * Which keys a query sees (the additive 0 / -inf mask of the Flash Attention
 * 2 page, "Causal masking", Option A, with the key tiles the mask removes
 * entirely skipped): in a sequence of N_q queries and N_k keys, query i is
 * aligned with key i + off, off = N_k - N_q (the last query with the last
 * key), and sees key j (0 <= j < N_k) iff
 *
 *     j < prefix_len,  or
 *     i + off - window_left <= j <= i + off + window_right
 *
 * where a window of -1 is unbounded on that side.  So (-1, -1) is full
 * attention, (-1, 0) causal (j <= i when N_q = N_k), (w, 0) a sliding window
 * of the w keys before each query and itself, and (-1, 0) with prefix_len = P
 * a prefix-LM (the first P keys visible to every query).  A query that sees
 * no key gets O = 0 and LSE = -inf.
 *
 * Element (b, h, i, c) of a tensor X in {q, o} is at
 *   X + b*X_strides[0] + h*X_strides[1] + (r0 + i)*X_strides[2] + c
 * elements, and of k, v likewise with key rows; lse (b, h, i) is at
 *   lse + b*lse_strides[0] + h*lse_strides[1] + (r0 + i).
 * Unpacked batches: r0 = 0, i < seqlen_q, j < seqlen_k.  Packed batches
 * (cu_seqlens_q and cu_seqlens_k both set): sequence b's query rows are
 * cu_seqlens_q[b] <= r < cu_seqlens_q[b+1] of q/o/lse (r0 = cu_seqlens_q[b])
 * and its keys cu_seqlens_k[b] <= r < cu_seqlens_k[b+1] of k/v; the batch
 * strides are ignored.
 */
typedef struct fa2_fwd_params {
  const void* q;          /* device, `dtype`, 16-byte aligned; read only */
  const void* k;          /* device, `dtype`, 16-byte aligned; read only */
  const void* v;          /* device, `dtype`, 16-byte aligned; read only */
  void* o;                /* device, `dtype`, 16-byte aligned; written */
  float* lse;             /* device, float32, 4-byte aligned; written (natural log) */
  int batch;              /* B >= 1 (packed: number of sequences) */
  int heads;              /* H >= 1 */
  int seqlen_q;           /* N_q >= 1 (packed: the longest sequence's query count) */
  int seqlen_k;           /* N_k >= 1 (packed: ignored) */
  int head_dim;           /* d: 64, 128 or 256 */
  int dtype;              /* FA2_FP16 or FA2_BF16 */
  float scale;            /* any finite value */
  int window_left;        /* >= 0, or -1 = unbounded */
  int window_right;       /* >= 0, or -1 = unbounded */
  int prefix_len;         /* >= 0 */
  int64_t q_strides[3];   /* batch, head, row strides in elements; multiples of 8 */
  int64_t k_strides[3];   /*   (a stride of a dimension of size 1 is ignored) */
  int64_t v_strides[3];
  int64_t o_strides[3];
  int64_t lse_strides[2]; /* batch, head strides in elements (row stride 1); >= 0 */
  const int* cu_seqlens_q; /* device, [batch + 1] int32 row offsets, or NULL */
  const int* cu_seqlens_k; /* device, [batch + 1] int32 row offsets, or NULL */
  int total_q;            /* packed: rows of q, o and lse (>= 1); else ignored */
  int total_k;            /* packed: rows of k and v (>= 1); else ignored */
} fa2_fwd_params;

/* sizeof(fa2_fwd_params) as compiled into the library (binding check). */
size_t fa2_fwd_params_size(void);

/*
 * fa2_fwd_ex -- the forward pass for fa2_fwd_params (asynchronous on
 * `stream`).  Same arithmetic and kernels as fa2_fwd, which is the special
 * case of contiguous [B,H,N,d] tensors, N_q = N_k = N, no prefix and
 * window (-1, causal ? 0 : -1).
 *
 * Checks before any launch: sizes, dtype, head dim, scale and windows as
 * documented above (FA2_ERR_INVALID_ARG / FA2_ERR_UNSUPPORTED); pointers
 * non-null and aligned and strides of dimensions larger than 1 positive
 * multiples of 8 elements below 2^39 (FA2_ERR_MISALIGNED for alignment,
 * FA2_ERR_INVALID_ARG otherwise); the byte ranges o and lse can touch
 * overlap neither each other nor those of q, k and v (FA2_ERR_INVALID_ARG);
 * only one of cu_seqlens_q / cu_seqlens_k set (FA2_ERR_INVALID_ARG).  The
 * caller keeps o's elements distinct (no two (b,h,i,c) at one address).
 *
 * Packed offsets live on the device and are checked by the kernel: a
 * sequence with cu_seqlens_q[b] > cu_seqlens_q[b+1], an offset outside
 * [0, total_q] (or [0, total_k] for keys), or more than seqlen_q queries is
 * left unwritten and the next fa2_get_device_status returns
 * FA2_ERR_DEVICE_SEQLENS.  The other sequences are written, except where
 * such offsets make in-range sequences' query rows overlap: a batch of at
 * most 192 sequences launches one CTA per real 128-row tile (as many as
 * non-overlapping sequences can hold), and tiles past that are skipped.
 * Rows of k and v outside a sequence may be read
 * (key tiles are 128 rows) and are multiplied by P = 0, so they must hold
 * finite values; rows past total_k read as zero.  Deterministic.
 */
int fa2_fwd_ex(const fa2_fwd_params* params, void* stream);

/* Query rows per sequence fa2_decode takes. */
#define FA2_DECODE_MAX_Q 8

/*
 * fa2_decode -- the forward pass for few query rows against many keys (the
 * decoding regime: a new token, or up to FA2_DECODE_MAX_Q of them, attending
 * to a long key/value cache).  Lesson 6.6 ("Common misconceptions") notes
 * that single-row decoding needs its own kernel: with one query row there is
 * no tile to fill a tensor core and the step is bound by reading K and V.
 * The keys of each (batch, head) are split into chunks reduced by separate
 * CTAs to online-softmax states (m, l, O~) that a second kernel merges with
 * the rescaling step of the tiled loop (Lesson 6.6, "Online softmax").
 * At d = 128 (and at d = 64 from two query rows on) the tiled tensor-core
 * kernel reduces each chunk for the whole query tile; one row at d = 64, and
 * d = 256, run the chunks on CUDA cores.
 *
 * Arguments as fa2_fwd_ex (same struct, masks, strides and packed batches),
 * with seqlen_q <= FA2_DECODE_MAX_Q (FA2_ERR_UNSUPPORTED otherwise; packed:
 * every sequence's query count) and seqlen_k the key count (packed: the
 * longest sequence's key count -- it sizes the split grid, which covers at
 * least that many keys; a sequence with more keys than the grid covers is
 * left unwritten and reported as FA2_ERR_DEVICE_SEQLENS).
 * `workspace`: device, >= fa2_decode_workspace_bytes(params) bytes, 256-byte
 * aligned, owned by the caller, overlapping no tensor; it holds fp32 partial
 * states and is written before it is read.  Asynchronous on `stream`; two
 * kernel launches (one when the keys fit a single chunk on the tensor-core
 * path).  Deterministic.
 */
int fa2_decode(const fa2_fwd_params* params, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace fa2_decode needs for these sizes (0 if they are invalid); it does
 * not depend on the device. */
size_t fa2_decode_workspace_bytes(const fa2_fwd_params* params);

/*
 * fa2_fwd_host -- the same forward pass on HOST buffers, end to end.
 *
 * Copies q, k, v (host, [B,H,N,d] `dtype`; pinned memory gives full copy
 * bandwidth) into the caller's device workspace, runs fa2_fwd on `stream`,
 * copies o and lse back into the host buffers and synchronises before
 * returning.  `workspace` is a device buffer of at least
 * fa2_fwd_host_workspace_bytes(B,H,N,d) bytes, 256-byte aligned, owned by the
 * caller.  Returns FA2_ERR_DEVICE_TIMEOUT if a kernel wait timed out.
 *
 * Problems with at least 48 MB of input are cut into up to 8 groups of
 * (b,h) slices: the copy-in of the next group and the copy-out of the
 * previous one run on two copy streams the library creates once per device
 * while the forward pass of the current group runs on `stream` (which first
 * waits for work already queued on it).  Such calls on one device are
 * serialised by the library.  Results are identical to the unsplit pass.
 */
int fa2_fwd_host(const void* q_host, const void* k_host, const void* v_host, void* o_host,
                 float* lse_host, void* workspace, size_t workspace_bytes,
                 int B, int H, int N, int d, float scale, int causal, int dtype, void* stream);

/* Device workspace fa2_fwd_host needs: q, k, v, o and lse, each 256-byte aligned. */
size_t fa2_fwd_host_workspace_bytes(int B, int H, int N, int d);

/* Bytes of the library's static device scratch used by fa2_fwd_host_noalloc. */
#define FA2_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)

/*
 * fa2_fwd_host_noalloc -- fa2_fwd_host for callers that cannot allocate
 * device memory.  The pages have no counterpart: it exists for callers that
 * hold only host buffers and are not allowed to call cudaMalloc -- e.g. a
 * process whose device memory is wholly reserved by another allocator, so a
 * raw cudaMalloc would fail, or a latency-bound loop that must not call an
 * allocator that may synchronise the device.
 *
 * Same arguments and results as fa2_fwd_host, without the workspace: the
 * device staging copies of q, k, v, o and lse live in one static device
 * array of FA2_NOALLOC_SCRATCH_BYTES bytes that the library defines, which
 * every GPU that loads the library holds until the process exits.  The call
 * allocates nothing (no cudaMalloc or cudaFree, no allocating library call).
 *
 *   Limit: fa2_fwd_host_workspace_bytes(B, H, N, d) must not exceed
 *   FA2_NOALLOC_SCRATCH_BYTES; larger problems return FA2_ERR_SCRATCH_LIMIT
 *   before any CUDA call.
 *
 * The first call on a device looks up the array's device address on that
 * device (with it current); make that first call before any stream capture.
 * All calls on a device share the one array: calls whose work overlaps on
 * the GPU (other streams, other host threads) race and must be serialised by
 * the caller.  Nothing in the array needs to start at zero -- every byte a
 * call reads was written earlier in that same call.  The call synchronises
 * `stream` before returning.
 */
int fa2_fwd_host_noalloc(const void* q_host, const void* k_host, const void* v_host, void* o_host,
                         float* lse_host, int B, int H, int N, int d, float scale, int causal, int dtype,
                         void* stream);

/*
 * fa2_get_device_status -- synchronises `stream`, then returns and clears the
 * current device's status word: FA2_OK, FA2_ERR_DEVICE_TIMEOUT if some
 * kernel's bounded wait on an mbarrier gave up (the kernel then abandoned its
 * tile, released its tensor memory and returned instead of hanging), else
 * FA2_ERR_DEVICE_SEQLENS if fa2_fwd_ex met out-of-range packed offsets, else
 * FA2_ERR_DEVICE_PAGES if a paged-cache call met lengths, a slot or a page out
 * of range.
 * `detail` (may be NULL) receives the raw status bits (role and wait site).
 */
int fa2_get_device_status(void* stream, uint32_t* detail);

/*
 * fa2_bwd -- gradients of fa2_fwd for an upstream gradient dout
 * (FlashAttention V2 in depth, section 7: P = exp(S - L) rebuilt from the
 * forward's logsumexp, dV = P^T dO, dP = dO V^T, D_i = rowsum(dO_i o O_i),
 * dS = P o (dP - D), dQ = scale dS K, dK = scale dS^T Q).  Asynchronous on
 * `stream`.
 *
 *   q, k, v, o, dout : device, [B,H,N,d] `dtype` (o is fa2_fwd's output)
 *   lse              : device, [B,H,N] float32, fa2_fwd's logsumexp
 *   dq, dk, dv       : device, [B,H,N,d] `dtype`, written
 *   workspace        : device, >= fa2_bwd_workspace_bytes(B,H,N,d) bytes,
 *                      256-byte aligned, owned by the caller: an fp32 dQ
 *                      accumulator [B,H,N,d] and D [B,H,N], both written
 *                      before they are read
 *   d                : 64, 128 or 256 (at d = 256 each 128-key tile runs as two
 *                      CTAs, one per half of the head dimension, that both
 *                      rebuild the tile's S and dP)
 *   other arguments  : as fa2_fwd
 *
 * dK and dV are each written once; dQ is accumulated over key tiles with
 * fp32 reduce-adds in L2 (TMA), so its last bits may vary between runs.
 * Outputs and workspace must not overlap any input or each other.  This is
 * fa2_bwd_ex for contiguous tensors and window (-1, causal ? 0 : -1).
 */
int fa2_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dout,
            void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes,
            int B, int H, int N, int d, float scale, int causal, int dtype, void* stream);

/* Device workspace fa2_bwd needs: fp32 [B,H,N,d] + fp32 [B,H,N], each 256-byte aligned. */
size_t fa2_bwd_workspace_bytes(int B, int H, int N, int d);

/*
 * fa2_bwd_params / fa2_bwd_ex -- gradients of fa2_fwd_ex: the same masks
 * (band, prefix), unequal query / key lengths, strided layouts and packed
 * batches.  `fwd` holds the forward call's arguments (q, k, v; o and lse
 * are the forward's outputs and are read here); the gradients share the
 * layouts of their primal tensors: dout and dq/dk/dv use o's, q's, k's and
 * v's strides.  head_dim 64, 128 or 256 (FA2_ERR_UNSUPPORTED otherwise).  Packed
 * batches: fwd.seqlen_k is the longest sequence's key count (it sizes the
 * grid; a sequence with more keys is left unwritten and reported as
 * FA2_ERR_DEVICE_SEQLENS; out-of-range offsets behave as in fa2_fwd_ex,
 * with key tiles in place of query tiles), and rows of dq outside every
 * sequence are set to
 * zero.  A key no query row sees gets dK = dV = 0; a query row that sees no
 * key gets dQ = 0.
 *
 * `workspace`: device, >= fa2_bwd_ex_workspace_bytes(&fwd) bytes, 256-byte
 * aligned: the fp32 dQ accumulator and D per row of every (batch, head)
 * slice, written before read.  dq, dk, dv and the workspace overlap no input
 * and no other output.  Asynchronous on `stream` (three kernels); dQ is
 * accumulated with fp32 reduce-adds, so its last bits may vary between runs.
 */
typedef struct fa2_bwd_params {
  fa2_fwd_params fwd;
  const void* dout;       /* device, o's layout, 16-byte aligned */
  void* dq;               /* device, q's layout, written */
  void* dk;               /* device, k's layout, written */
  void* dv;               /* device, v's layout, written */
  void* workspace;
  size_t workspace_bytes;
} fa2_bwd_params;

size_t fa2_bwd_ex_workspace_bytes(const fa2_fwd_params* fwd);
int fa2_bwd_ex(const fa2_bwd_params* params, void* stream);

/*
 * fa2_paged_cache -- a key/value cache in pages of page_size rows, shared by
 * the requests of a server: element (page, head, row, c) of k is at
 *   k + page*k_strides[0] + head*k_strides[1] + row*k_strides[2] + c
 * elements, v likewise.  So [num_pages, heads, page_size, d] and [num_pages,
 * page_size, heads, d] storage both fit, and k and v may interleave in one
 * allocation (fa2_paged_append: their elements are distinct).  Row r of page p
 * is slot p * page_size + r.  Strides of dimensions larger than 1 are positive
 * multiples of 8 elements below 2^39.
 */
typedef struct fa2_paged_cache {
  void* k;                /* device, `dtype`, 16-byte aligned; written by fa2_paged_append only */
  void* v;                /* device, `dtype`, 16-byte aligned; written by fa2_paged_append only */
  int64_t k_strides[3];   /* page, head, row strides in elements */
  int64_t v_strides[3];
  int num_pages;          /* >= 1; num_pages * page_size < 2^31 (FA2_ERR_UNSUPPORTED) */
  int page_size;          /* 8, 16, 32 or a multiple of 64 (FA2_ERR_UNSUPPORTED otherwise) */
  int heads;              /* K/V heads, 1 .. 65536 (FA2_ERR_UNSUPPORTED above) */
  int head_dim;           /* d: 64, 128 or 256 */
  int dtype;              /* FA2_FP16 or FA2_BF16 */
} fa2_paged_cache;

/*
 * fa2_paged_plan -- block tables and the slot map of one serving step, built
 * on the GPU from the requests' lengths.  Request b holds context_lens[b]
 * cached tokens, on the first ceil(context / page_size) entries of its block
 * table row, and gets query_lens[b] new ones (0: idle).  The call
 *   - sets cu_seqlens_q (exclusive prefix sums of query_lens, batch + 1) and
 *     seqlens_k[b] = context_lens[b] + query_lens[b];
 *   - takes the pages the new tokens need beyond those held from the top of
 *     the stack free_pages[0 .. *free_count), in order of the requests and of
 *     each request's pages (the first page taken is free_pages[*free_count -
 *     1]), and writes them to the table rows; other entries are left;
 *   - sets slots[t] of new token t (packed order) to its slot, and to -1 for
 *     the rows of slots behind the last token (padding);
 *   - sets *free_left to what remains of the stack.
 * free_count is read, not written, so the call may be repeated; the next step
 * passes free_left as its free_count.
 *
 * A step that cannot be placed -- a negative length, a request past max_pages
 * pages, more tokens than total_q, more pages than *free_count, *free_count
 * outside [0, num_free] -- is refused whole: cu_seqlens_q = seqlens_k = 0,
 * slots = -1, *free_left = *free_count, the table as it was (so an append and
 * a forward of that step write nothing), and the next fa2_get_device_status
 * returns FA2_ERR_DEVICE_PAGES.  The same status reports a page outside [0,
 * num_pages) met in the free list or in a held entry; its tokens get slot -1.
 *
 * One kernel, asynchronous on `stream`, deterministic, no workspace.  Outputs
 * overlap neither each other nor an input (FA2_ERR_INVALID_ARG).  Checks as
 * fa2_fwd_ex; batch <= FA2_PAGED_PLAN_MAX_BATCH (FA2_ERR_UNSUPPORTED).
 */
#define FA2_PAGED_PLAN_MAX_BATCH 16384

typedef struct fa2_paged_plan_params {
  const int* context_lens; /* device, [batch] int32 */
  const int* query_lens;   /* device, [batch] int32 */
  const int* free_pages;   /* device, [num_free] int32 (may be NULL when num_free = 0) */
  const int* free_count;   /* device, one int32 */
  int* block_table;        /* device, [batch][max_pages] int32, rows table_stride apart; updated */
  int* cu_seqlens_q;       /* device, [batch + 1] int32; written */
  int* seqlens_k;          /* device, [batch] int32; written */
  int* slots;              /* device, [total_q] int32; written */
  int* free_left;          /* device, one int32; written */
  int64_t table_stride;    /* elements; >= max_pages unless batch = 1 */
  int batch;               /* >= 1 */
  int max_pages;           /* table entries per request >= 1; max_pages * page_size <= 2^31 - 4096 */
  int num_pages;           /* pages of the cache >= 1; num_pages * page_size < 2^31 */
  int page_size;           /* >= 1 */
  int total_q;             /* rows of slots >= 1: the step's tokens, with padding */
  int num_free;            /* entries of free_pages >= 0 */
} fa2_paged_plan_params;

int fa2_paged_plan(const fa2_paged_plan_params* params, void* stream);

/*
 * fa2_paged_append -- new key/value rows into a paged cache: row t of k and v
 * ([total, heads, d] by strides: token, head) goes to slot slots[t] of every
 * head, bit for bit.  A negative slot is skipped (padding); a slot past the
 * cache is skipped and reported (FA2_ERR_DEVICE_PAGES).  The slots >= 0 of one
 * call are distinct (as fa2_paged_plan's are): which of two rows with one slot
 * remains is not determined, per 16 bytes.  Other rows of the cache are not
 * touched.  k, v and slots overlap neither cache tensor.  One kernel,
 * asynchronous on `stream`.
 */
typedef struct fa2_paged_append_params {
  fa2_paged_cache cache;
  const void* k;           /* device, cache.dtype, 16-byte aligned; read only */
  const void* v;           /* device, cache.dtype, 16-byte aligned; read only */
  const int* slots;        /* device, [total] int32 */
  int64_t k_strides[2];    /* token, head strides in elements; multiples of 8 */
  int64_t v_strides[2];
  int total;               /* rows >= 1 */
} fa2_paged_append_params;

int fa2_paged_append(const fa2_paged_append_params* params, void* stream);

/*
 * fa2_paged_fwd -- attention of each sequence's query tokens (one while
 * decoding, a chunk of a prompt, or any mix over the batch) over its keys in a
 * paged cache.  Sequence b's queries are rows cu_seqlens_q[b] <= r <
 * cu_seqlens_q[b+1] of q / o ([total_q, heads, d] by strides: token, head) and
 * of lse ([heads, total_q], head stride lse_stride); its seqlens_k[b] keys --
 * the new tokens' own among them, already appended -- are rows j % page_size
 * of pages block_table[b][j / page_size].  Query head i reads K/V head i /
 * (heads / cache.heads); heads is a multiple of cache.heads, at most 128 times
 * it (FA2_ERR_UNSUPPORTED).  Masks, scale and rows that see no key (O = 0, LSE =
 * -inf) as fa2_fwd_ex: causal attention is window (-1, 0).
 * Beside the prefix, which every query sees whole, also ahead of itself, there
 * are sink keys: query i also sees key j iff
 *
 *     j < sink_len  and  j <= i + off + window_right
 *
 * (window_right = -1: any j < sink_len), so a sliding window that keeps the
 * first s keys in sight is (w, 0) with sink_len = s.  Without a left window
 * the sinks are in the band already.  P is rounded to 16 bits for the product
 * with the values; in bf16 its low part is added on tiles of 64 keys that the
 * mask cuts, and on all tiles of a query tile (128 / group tokens) that visits
 * at most three.  Sums are fp32; a batch decides where a sequence's keys are
 * cut into partial sums, so the same sequence may differ in its last bits in
 * another batch or under another max_seqlen_q.
 *
 * Rows of q / o / lse outside every sequence are left as they were.  Keys no
 * query row of a sequence sees (rows past its length, keys before a window)
 * may hold anything, NaN included, and their table entries are not read.  A NaN
 * in a query row or in a key that it sees makes the row's O and LSE NaN, a NaN
 * in a value that it sees that column of O (and it may that column in other rows
 * of the sequence); queries and visible keys and values are not infinite.
 *
 * Lengths, offsets and tables live on the device and are checked by the
 * kernel: a sequence with cu_seqlens_q[b] > cu_seqlens_q[b+1], an offset
 * outside [0, total_q], more than max_seqlen_q queries, or seqlens_k[b]
 * outside [0, max_pages * page_size] is left unwritten and reported as
 * FA2_ERR_DEVICE_SEQLENS (sequences whose query rows overlap: as fa2_fwd_ex).
 * A needed page outside [0, num_pages) reads as zero keys and values and is
 * reported as FA2_ERR_DEVICE_PAGES.
 *
 * `workspace`: device, >= fa2_paged_fwd_workspace_bytes(params) bytes, 256-byte
 * aligned, overlapping no tensor: fp32 partial states, written before they
 * are read (calls that overlap on the GPU each need their own).  o, lse and
 * the workspace overlap nothing else.  Asynchronous on `stream`, two kernels;
 * the host reads no length, so a captured call replays with new lengths,
 * tables and slots in the same buffers.  Deterministic.  The first call on a
 * device comes before any stream capture.
 */
typedef struct fa2_paged_params {
  fa2_paged_cache cache;
  const void* q;           /* device, cache.dtype, 16-byte aligned; read only */
  void* o;                 /* device, cache.dtype, 16-byte aligned; written */
  float* lse;              /* device, float32; written (natural log) */
  const int* block_table;  /* device, [batch][max_pages] int32, rows table_stride apart */
  const int* cu_seqlens_q; /* device, [batch + 1] int32 */
  const int* seqlens_k;    /* device, [batch] int32 */
  int64_t table_stride;    /* elements; >= 0 (0: one row for all sequences) */
  int64_t q_strides[2];    /* token, head strides in elements; multiples of 8 */
  int64_t o_strides[2];
  int64_t lse_stride;      /* head stride in elements (token stride 1); >= total_q unless heads = 1 */
  int batch;               /* sequences >= 1 */
  int heads;               /* query heads >= 1 */
  int total_q;             /* rows of q, o and lse >= 1 */
  int max_seqlen_q;        /* longest sequence's query count >= 1 (sizes grid and workspace) */
  int max_pages;           /* table entries per sequence >= 1; max_pages * page_size <= 2^31 - 4096 */
  int window_left;         /* >= 0, or -1 = unbounded */
  int window_right;        /* >= 0, or -1 = unbounded */
  int prefix_len;          /* >= 0 */
  float scale;             /* any finite value */
  int sink_len;            /* >= 0 */
} fa2_paged_params;

/* sizeof(fa2_paged_params) as compiled into the library (binding check). */
size_t fa2_paged_params_size(void);

/* Workspace fa2_paged_fwd needs for these sizes (0 if they are invalid); it
 * depends on no length and not on the device. */
size_t fa2_paged_fwd_workspace_bytes(const fa2_paged_params* params);

int fa2_paged_fwd(const fa2_paged_params* params, void* workspace, size_t workspace_bytes, void* stream);

/*
 * fa2_selftest_wait_timeout -- exercises the kernels' failure path without a
 * GPU fault: launches one CTA whose single wait, made through the same
 * bounded-wait routine every forward-kernel wait uses, is on an mbarrier that
 * nothing ever completes.  After `limit_us` microseconds (1 .. 1e6) the wait
 * gives up, records its site in the device status word and the kernel
 * returns normally.  Asynchronous on `stream`; a following
 * fa2_get_device_status returns FA2_ERR_DEVICE_TIMEOUT (detail bit 8 + 11)
 * and clears the word.  No counterpart on the pages: it tests the library's
 * own hang protection (FlashAttention V2 in depth describes no failure
 * handling).
 */
int fa2_selftest_wait_timeout(int limit_us, void* stream);

/* Static English description of a status code. */
const char* fa2_status_string(int status);

/* Library version as major*10000 + minor*100 + patch. */
int fa2_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FA2_GB300_H */
