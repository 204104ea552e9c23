/*
 * ftd.h -- C ABI of the GB300 masked multi-head attention decode step.
 *
 * One call performs one decode step of masked multi-head attention for every
 * slot of a continuous batch, entirely in hand-written sm_103a kernels:
 *
 *   1. fused QKV bias add           q' = q + b_q, k' = k_new + b_k, v' = v_new + b_v
 *                                   (FasterTransformer practice notes, lpnh.cn,
 *                                   section 2.1: the projection output is split
 *                                   into Q/K/V and the bias is added in the fused
 *                                   attention kernel, with no extra HBM round trip)
 *   2. KV-cache append              K[b, h, L_b, :] = round(k'), V likewise
 *                                   (lpnh.cn section 2.2: a pre-allocated cache the
 *                                   new K/V is appended to at every token;
 *                                   "FasterTransformer source analysis",
 *                                   framerc.cn, section 3.2: one buffer sized for
 *                                   the preset maximum length, shared by offset)
 *   3. scores over the whole cache  s_t = scale * q' . K[t],  t = 0 .. L_b
 *   4. masked, stable softmax       p = softmax(s) over t <= L_b (the current
 *                                   position; nothing after it is visible)
 *   5. weighted sum                 o = sum_t p_t V[t]
 *   6. split-K merge                partial (max, sum, o) of several thread
 *                                   blocks combined by log-sum-exp ("10 tricks
 *                                   for Transformer throughput", pptc.cn,
 *                                   section 2.2: online softmax statistics, no
 *                                   N x N matrix in memory)
 *
 * with ragged per-slot lengths (intelliparadigm.com section 3.2, continuous
 * batching), grouped / multi-query heads (pptc.cn section 3.4: query head h
 * reads kv head h / (Hq / Hkv)) and an INT8 cache with an fp32 scale per
 * (slot, kv head, position) (pptc.cn section 3.1).
 *
 * Four options the pages name next to the step:
 *  - out_dtype F16 / BF16: the output is rounded once, to nearest even, from
 *    the fp32 result, in the precision the following projection reads
 *    (lpnh.cn section 2.1: the fused kernels run in half precision).
 *  - window W > 0: sliding-window attention, slot b attends to positions
 *    max(0, L_b + 1 - W) .. L_b only (pptc.cn section 3.1: keep only the
 *    recent part of the history in the cache).
 *  - page_size > 0: a paged cache (intelliparadigm.com section 5.1: the cache
 *    cut into fixed pages, e.g. 256 tokens each; framerc.cn section 3.2:
 *    fixed-size blocks mapped like a virtual-memory page table): the cache is
 *    a pool of pages and a per-slot block table maps positions to pages;
 *    served by ftd_decode_mha_paged.
 *  - q_len T > 1: T new tokens per slot in one step, as a speculative
 *    verification pass checks a run of draft tokens (pptc.cn section 4.3).
 *    Token j of slot b is appended at position L_b + j and its query attends
 *    to positions 0 .. L_b + j (with a window, the last W of them).  The
 *    caller then advances seq_lens[b] by the number of tokens it accepts;
 *    rows written past that are overwritten by the next step.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - B = max_batch, Hq = n_q_heads, Hkv = n_kv_heads, D = head_dim,
 *    Lmax = max_len.  L_b = seq_lens[b] is the number of tokens already in
 *    the cache for slot b; the new token is written at position L_b and
 *    attends to positions 0 .. L_b inclusive.
 *  - Layouts are dense and row-major (T = q_len, 1 unless set):
 *        q      [B][T][Hq][D]     qkv dtype
 *        k_new  [B][T][Hkv][D]    qkv dtype      v_new likewise
 *        bias   [(Hq + 2*Hkv)*D]  qkv dtype, the q part, then k, then v
 *        cache  [B][Hkv][Lmax][D] cache dtype    (k_cache, v_cache)
 *        scales [2][B][Hkv][Lmax] fp32, plane 0 for K and plane 1 for V
 *                                 (INT8 caches only)
 *        out    [B][T][Hq][D]     out_dtype (fp32 unless the config says)
 *    A paged context replaces the cache and scale layouts by
 *        pages  [num_pages][Hkv][page_size][D]  cache dtype (k_pages, v_pages)
 *        scales [2][num_pages][Hkv][page_size]  fp32 (INT8 caches only)
 *        block_table [B][ceil(Lmax / page_size)] int32: entry i of slot b is
 *               the page holding positions i*page_size .. (i+1)*page_size - 1.
 *  - Slots with seq_lens[b] < 0 are inactive: their cache is untouched and
 *    their output is zero.  seq_lens[b] + T > Lmax is an overflow: the slot is
 *    skipped the same way and a sticky device error is raised, which
 *    ftd_get_error() reports as FTD_ERR_SEQ_OVERFLOW.  Nothing traps.
 *  - Device pointers must be 16-byte aligned.  All device work goes to the
 *    caller's stream (a cudaStream_t passed as void*; NULL = legacy default
 *    stream) and is asynchronous; the decode entry points never allocate.
 *  - The caller advances seq_lens after a step; the library never writes it.
 *  - Errors found on the host return synchronously and leave the device
 *    untouched.  ftd_last_error() describes the most recent one.
 */
#ifndef FTD_H
#define FTD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FTD_OK = 0,
    FTD_ERR_INVALID_ARG = 1,     /* null pointer, bad size, misaligned pointer */
    FTD_ERR_UNSUPPORTED = 2,     /* dtype / head_dim combination not built */
    FTD_ERR_OOM = 3,             /* ftd_init could not allocate its pool */
    FTD_ERR_CUDA = 4,            /* a CUDA runtime call failed */
    FTD_ERR_SEQ_OVERFLOW = 5,    /* some seq_lens[b] + q_len > max_len in a past call */
    FTD_ERR_DEVICE_TIMEOUT = 6,  /* a kernel gave up waiting for a copy (bounded wait) */
    FTD_ERR_BAD_PAGE = 7         /* in a past call a block-table entry was outside [0, num_pages), or a token's
                                    place or a count of free pages outside the cache (ftd_norm_rope_qkv, ftd_build_tables) */
} ftd_status;

typedef enum { FTD_F32 = 0, FTD_F16 = 1, FTD_BF16 = 2, FTD_I8 = 3 } ftd_dtype;

typedef struct {
    int max_batch;       /* B, 1 .. 1024 */
    int n_q_heads;       /* Hq, a multiple of n_kv_heads */
    int n_kv_heads;      /* Hkv >= 1 (Hkv == Hq: MHA, Hkv == 1: MQA) */
    int head_dim;        /* D: 64 or 128 */
    int max_len;         /* Lmax: a multiple of 16 */
    ftd_dtype qkv_dtype;   /* q, k_new, v_new, bias: F32, F16 or BF16 */
    ftd_dtype cache_dtype; /* F32, F16, BF16 or I8 */
    float softmax_scale;   /* 0 selects 1/sqrt(head_dim) */
    /* Options; an all-zero tail gives the plain step (fp32 out, full context,
     * contiguous cache). */
    ftd_dtype out_dtype;   /* F32 (0), F16 or BF16 */
    int window;            /* 0: whole context; W > 0: the last W positions */
    int page_size;         /* 0: contiguous cache; else a power of two >= 128 */
    int num_pages;         /* pages in the pool when page_size > 0 */
    int q_len;             /* new tokens per slot per step, 0 or 1 .. 64 (0 = 1) */
    int kernel;            /* FTD_KERNEL_AUTO (0): the library's choice;
                              FTD_KERNEL_CUDA_CORE (1): the CUDA-core split-K kernel
                              for every configuration (the tensor-core kernel is
                              otherwise taken for head_dim 128 caches whose kv heads
                              carry a multiple of 4 query rows, 8 for INT8) */
    int proj_dim;          /* 0: no output projection; F > 0 (a multiple of 128): the
                              context also serves ftd_decode_mha_proj, y = out . W_o^T
                              with W_o [F][n_q_heads * head_dim] (F16 / BF16 qkv only) */
    int wait_limit_us;     /* 0: a kernel's bounded waits give up after about 2 s;
                              else after this many microseconds (measured in SM clock
                              cycles at the device's peak clock), raising
                              FTD_ERR_DEVICE_TIMEOUT.  The drain of copies still in
                              flight after such an abort always keeps the 2 s limit. */
} ftd_config;

enum { FTD_KERNEL_AUTO = 0, FTD_KERNEL_CUDA_CORE = 1 };

typedef struct ftd_ctx ftd_ctx;

/*
 * ftd_init -- validate cfg and pre-allocate the cache pool.
 * One cudaMalloc on the current device holds the K and V caches (zeroed; for
 * a paged context, num_pages pages of each),
 * the INT8 scale planes, the split-K workspace, the sticky error word and the
 * staging buffers of ftd_decode_mha_host.  Zeroing runs on `stream`.
 * The pool is the pre-allocated buffer of framerc.cn section 3.2 (allocated
 * once for max_batch x max_len, requests share it by offset, no resize).
 * On success *out owns the pool until ftd_destroy.  Returns INVALID_ARG,
 * UNSUPPORTED, OOM or CUDA on failure, with *out set to NULL.
 */
ftd_status ftd_init(const ftd_config* cfg, void* stream, ftd_ctx** out);

/*
 * ftd_cache_ptrs -- device addresses of the context's own pool: the K and V
 * caches [B][Hkv][Lmax][D] (pages for a paged context) and the INT8 scale
 * planes, i.e. the per-sequence cache pointers of the decoding state that
 * intelliparadigm.com section 3.2 keeps for each request, and the buffer that
 * framerc.cn section 3.2 pre-allocates once.  Any output pointer may be NULL.
 * *scales is NULL unless the cache is INT8.  The caller may fill the cache
 * (prefill) through these pointers.  Returns INVALID_ARG for a NULL ctx.
 */
ftd_status ftd_cache_ptrs(ftd_ctx* ctx, void** k_cache, void** v_cache, float** scales);

/*
 * ftd_decode_mha -- one decode step for all max_batch slots (device buffers).
 *   q, k_new, v_new : device, caller-owned, qkv dtype, layouts above.
 *   qkv_bias        : device or NULL (no bias).
 *   k_cache, v_cache: device caches with the layout above, read and appended
 *                     to in place; NULL selects the context's own pool.
 *   seq_lens        : device int32 [B]; read only.
 *   scales          : device fp32 [2][B][Hkv][Lmax] for INT8 caches (NULL
 *                     selects the pool's planes); ignored otherwise.
 *   out             : device [B][T][Hq][D] of out_dtype; every element is written.
 *   stream          : cudaStream_t as void*.
 * Launches one kernel; no host synchronisation and no allocation.  Two calls
 * on the same context must not overlap in time (they share the workspace):
 * issue them on one stream, or order their streams with events.
 * The kernel is launched with programmatic dependent launch: it may start
 * while the preceding kernel on the stream finishes, if that kernel allows
 * it (this library's decode kernels do, right after their own start).  Before
 * it waits for that kernel it reads only seq_lens, to plan its work and to
 * prefetch cache lines into L2 (always safe); after the wait it reads seq_lens
 * again and re-plans if they changed, so a preceding kernel may write seq_lens
 * (for example the caller's seq_lens += accepted kernel).
 * A paged context (page_size > 0) is refused with INVALID_ARG.
 */
ftd_status ftd_decode_mha(ftd_ctx* ctx, const void* q, const void* k_new, const void* v_new,
                          const void* qkv_bias, void* k_cache, void* v_cache,
                          const int32_t* seq_lens, float* scales, void* out, void* stream);

/*
 * ftd_decode_mha_current -- ftd_decode_mha with the specified ten-argument
 * signature (no context handle): it runs on the most recently initialised
 * context that has not been destroyed (destroying it makes the one initialised
 * before it current again), and returns FTD_ERR_INVALID_ARG when there is
 * none.  It holds a library lock while it launches, so an ftd_destroy in
 * another thread waits for it.  For a process that holds one context; with
 * several, pass the handle to ftd_decode_mha instead.
 */
ftd_status ftd_decode_mha_current(const void* q, const void* k_new, const void* v_new, const void* qkv_bias,
                                  void* k_cache, void* v_cache, const int32_t* seq_lens, float* scales,
                                  void* out, void* stream);

/*
 * ftd_decode_mha_paged -- ftd_decode_mha over a paged cache (intelliparadigm.com
 * section 5.1, framerc.cn section 3.2: the cache is cut into fixed-size pages
 * and a block table maps each slot's positions to pages, so the pool holds
 * the pages in use rather than max_batch x max_len).
 *   k_pages, v_pages: device pages [num_pages][Hkv][page_size][D]; NULL
 *                     selects the context's own pool.
 *   block_table     : device int32 [B][ceil(max_len / page_size)], read only;
 *                     only entries covering positions 0 .. L_b of active
 *                     slots are read (the window start's page and on, when a
 *                     window is set).  The new token goes to position L_b of
 *                     its page.  Pages must not be shared between the
 *                     positions that two slots write.
 *   scales          : device fp32 [2][num_pages][Hkv][page_size] (INT8), NULL
 *                     selects the pool's planes.
 * Other arguments as in ftd_decode_mha.  An entry outside [0, num_pages)
 * raises a sticky device error (FTD_ERR_BAD_PAGE from ftd_get_error); the
 * kernel then reads nothing through it and writes no cache row for it, and
 * the output of that slot is undefined.  Refused (INVALID_ARG) on a context
 * without pages.
 */
ftd_status ftd_decode_mha_paged(ftd_ctx* ctx, const void* q, const void* k_new, const void* v_new,
                                const void* qkv_bias, void* k_pages, void* v_pages,
                                const int32_t* block_table, const int32_t* seq_lens, float* scales,
                                void* out, void* stream);

/*
 * ftd_decode_mha_proj -- ftd_decode_mha followed, in the same call and on the
 * same stream, by the output projection of the step's result (the fused
 * kernels hand their output straight to the next projection in half
 * precision, "FasterTransformer practice", lpnh.cn, section 2.1):
 *     y[b][t][f] = sum_k W_o[f][k] * out[b][t][k],   k < n_q_heads * head_dim,
 * out taken as stored (its out_dtype) and flattened over heads.  The decode
 * kernel's final stores also write each output value as a high and a low half
 * of W_o's type into two planes of the context, so the product keeps about 16
 * mantissa bits of an fp32 out; a second kernel, a tcgen05 GEMM that reads W_o
 * once, starts while the decode kernel's last blocks finish (programmatic
 * dependent launch) and writes y.
 *   w_o : device [proj_dim][n_q_heads * head_dim] in the qkv dtype (F16 or
 *         BF16; the layout of a linear layer's weight), 16-byte aligned, read only.
 *   y   : device [B][T][proj_dim] of out_dtype, 16-byte aligned; every element
 *         is written (zero for inactive and overflowing slots).
 * Other arguments as in ftd_decode_mha; out is written as well.  Needs a
 * context with proj_dim > 0 and a contiguous cache (INVALID_ARG otherwise).
 * Launches two kernels; no host synchronisation and no allocation.
 */
ftd_status ftd_decode_mha_proj(ftd_ctx* ctx, const void* q, const void* k_new, const void* v_new,
                               const void* qkv_bias, void* k_cache, void* v_cache, const int32_t* seq_lens,
                               float* scales, void* out, const void* w_o, void* y, void* stream);

/*
 * ftd_decode_mha_host -- the same step for callers whose per-step inputs live
 * in host memory (the host input-id update, kernel launches and device-to-host
 * read of the output that one decode step makes in lmnt.cn section 3.3).  q, k_new, v_new, qkv_bias (nullable), seq_lens and out are
 * HOST pointers; the caches stay on the device as in ftd_decode_mha (NULL =
 * the pool).  When every one of them is pinned, GPU-addressable memory
 * (cudaHostAlloc / cudaHostRegister; 16-byte aligned, seq_lens 4-byte) the
 * decode kernel reads the inputs in place and writes out straight into the
 * host buffer (one launch, no copy calls; on Grace systems both cross
 * NVLink-C2C).  The buffers must not change until the call returns.
 * Otherwise the inputs are copied in and out is copied back with
 * cudaMemcpyAsync.  Either way the call synchronises `stream` before it
 * returns, so out is valid on return.  Contiguous contexts only.
 */
ftd_status ftd_decode_mha_host(ftd_ctx* ctx, const void* q, const void* k_new, const void* v_new,
                               const void* qkv_bias, void* k_cache, void* v_cache,
                               const int32_t* seq_lens, float* scales, void* out, void* stream);

/*
 * ftd_get_error -- synchronise the stream of the context's last call, then
 * read and clear the sticky device error word.  A sequence that outgrows the
 * pre-allocated length is an error the caller must see, not a silent
 * overwrite (framerc.cn section 3.2; lmnt.cn section 5.2); the kernels skip
 * such a slot and set the word instead of trapping.  Returns FTD_OK,
 * FTD_ERR_SEQ_OVERFLOW, FTD_ERR_BAD_PAGE, FTD_ERR_DEVICE_TIMEOUT or
 * FTD_ERR_CUDA (the most serious first when several bits are set).  After a
 * timeout it also resets the split-K counters, so the next call starts clean.
 */
ftd_status ftd_get_error(ftd_ctx* ctx);

/* ftd_destroy -- free the pool (synchronises the device first).  NULL is a
 * no-op.  The context must not be in use by another thread's call; if it is
 * the current context of ftd_decode_mha_current, the most recently initialised
 * of the remaining live contexts becomes current. */
void ftd_destroy(ftd_ctx* ctx);

/* ftd_status_str -- static name of a status code. */
const char* ftd_status_str(ftd_status s);

/* ftd_last_error -- text of the most recent host-side error in this thread ("" if none). */
const char* ftd_last_error(void);

/* ftd_kernel_launches -- number of kernels this library has launched in this
 * process (every decode call adds one; host-side failures add none). */
uint64_t ftd_kernel_launches(void);

/*
 * ftd_debug_stall_next -- test hook for the bounded-wait error path; the pages
 * have no counterpart.  The next `calls` decode calls on ctx withhold the first
 * tile copy of block 0, so that block's waits run out after the context's
 * wait_limit_us, it drains what it has in flight and returns, and
 * ftd_get_error reports FTD_ERR_DEVICE_TIMEOUT (and resets the counters).
 * Outputs of such a call are undefined.  Nothing faults and nothing hangs:
 * every wait is bounded.  calls = 0 cancels.
 */
ftd_status ftd_debug_stall_next(ftd_ctx* ctx, int calls);

/*
 * ftd_debug_late_lengths -- test hook for the decode kernels' re-planning path;
 * the pages have no counterpart.  Launches, on `stream`, one small kernel that
 * at once allows the next launch on the stream to start (programmatic
 * dependent launch), waits about delay_us microseconds and then copies n int32
 * lengths from src to dst (both device pointers).  A decode call issued right
 * after it on the same stream with seq_lens = dst therefore plans its split
 * from the old lengths and must notice, after its wait, that they changed.
 * n is 1 .. 1024 and delay_us 0 .. 1e6; the kernel's wait is bounded by delay_us.
 */
ftd_status ftd_debug_late_lengths(const int32_t* src, int32_t* dst, int n, int delay_us, void* stream);

/*
 * ftd_debug_kernel -- test hook; the pages have no counterpart.  Which kernel an entry point takes on
 * ctx: entry 0 the step, 1 ftd_decode_mha_scored, 2 ftd_cross_mha.  *block_rows gets the query
 * rows of a block, *tensor_cores 1 or 0 (the CUDA cores); blocks of 32 and 64 rows on the
 * tensor cores are the wide kernel's.  Host work only.
 */
ftd_status ftd_debug_kernel(ftd_ctx* ctx, int entry, int* block_rows, int* tensor_cores);

/*
 * Operators around the step: rotary positions before it, alone or with norms of
 * the heads, block tables and slot maps from request lengths, the step that also
 * accumulates attention weights, the eviction by those weights, cross attention, and
 * the step of slots that share a prefix.  They take the context's shapes, types and caches, follow the
 * conventions above, launch on the caller's stream without allocating or
 * synchronising, and may be captured into a graph (after one call of
 * ftd_enable_scores, of ftd_enable_prefix, and of ftd_cross_mha, outside the capture).  Calls on one
 * context must not overlap in time, whichever entry points they are: graphs
 * captured from one context share its workspace too.
 */

enum { FTD_ROPE_HALVES = 0, FTD_ROPE_ADJACENT = 1 };
enum { FTD_ROPE_SECTIONS = 0, FTD_ROPE_INTERLEAVED = 1 };

typedef struct {
    int n_axes;       /* position axes (time, height, width, ...): 1 .. 4 */
    int rotary_dim;   /* R: the first R elements of a head turn, the others pass; even, 0 = head_dim */
    int section[4];   /* pairs that follow each axis; together R / 2 (one axis: 0 stands for R / 2) */
    int pairing;      /* FTD_ROPE_HALVES: pair i is elements (i, i + R/2); FTD_ROPE_ADJACENT: (2i, 2i + 1) */
    int order;        /* FTD_ROPE_SECTIONS: the first section[0] pairs follow axis 0, the next section[1] axis 1, ...;
                         FTD_ROPE_INTERLEAVED: pairs go to the axes in turn, an axis whose section is full is passed over */
    double theta;     /* pair i turns theta^(-2i/R) radians per position; 0 = 10000 */
    const double* inv_freq;  /* host, R / 2 radians per position that replace theta's; NULL: theta */
} ftd_rope_config;

/*
 * ftd_set_rope -- the rotary positions that ftd_rope_qkv applies on this context.
 * Copies what cfg holds (host work only); may be called again.  INVALID_ARG for
 * sizes that do not fit, leaving the previous setting.
 */
ftd_status ftd_set_rope(ftd_ctx* ctx, const ftd_rope_config* cfg);

/*
 * ftd_rope_qkv -- bias and rotary positions for n_tokens tokens, those of a step
 * (B * T in the order of q) or of a prompt, ahead of ftd_decode_mha (which is then
 * called without a bias) or of a cache fill:
 *   x = in + bias (one fp32 add);  for pair i, (a, b) of a query or key head, with
 *   w = positions[axis(i)][token] * inv_freq[i]:
 *   out_a = a cos w - b sin w,  out_b = b cos w + a sin w,
 * in fp32, rounded once to the qkv type.  Angles are wrapped exactly, so far
 * positions keep their full accuracy; positions may be negative.  Value heads only
 * take the bias.
 *   q, k, v   : device, qkv dtype; token t's heads at q + t * q_stride and k, v +
 *               t * kv_stride elements (0: dense rows), so a fused projection's
 *               [n][(Hq + 2 Hkv) * D] output is passed as three pointers into it.
 *               v and v_out may both be NULL.
 *   qkv_bias  : device [(Hq + 2 Hkv) * D] or NULL.
 *   positions : device int32 [n_axes][n_tokens].
 *   q_out, k_out, v_out : device, dense [n_tokens][Hq][D] and [n_tokens][Hkv][D]; each
 *               may be its own dense input.  Other overlaps are refused.
 * Pointers need the alignment of their elements.  The kernel moves 16 bytes at a time where
 * pointers and strides are 16-byte aligned and R / 2 is a multiple of 8 (fp32: 4), else the
 * half, quarter or eighth of that.
 * n_tokens 0 launches nothing.
 */
ftd_status ftd_rope_qkv(ftd_ctx* ctx, const void* q, const void* k, const void* v, int64_t q_stride,
                        int64_t kv_stride, const void* qkv_bias, const int32_t* positions, int64_t n_tokens,
                        void* q_out, void* k_out, void* v_out, void* stream);

/*
 * ftd_norm_rope_qkv -- ftd_rope_qkv with norms of the query and key heads ahead of the
 * rotation, and with keys and values that may go straight into the cache.  For a query or
 * key head x = in + bias whose kind has a weight w:
 *   y_e = x_e / sqrt(mean over the head of x^2 + eps) * (w_e + weight_offset),
 * then y turns as in ftd_rope_qkv (ftd_set_rope first); fp32 throughout, one rounding.
 *   q, k, v, q_stride, kv_stride, qkv_bias, positions, n_tokens, q_out : as in ftd_rope_qkv.
 *   q_weight, k_weight : device [D], qkv dtype, or NULL (no norm of that kind of head).
 *   eps       : finite, >= 0.   weight_offset : 0, or 1 for weights kept around zero.
 *   slots     : NULL: keys and values go to k_out, v_out as in ftd_rope_qkv, and the three
 *               cache arguments are NULL.  Else device int32 [n_tokens], a token's place in
 *               the cache: b * Lmax + position, on a paged context page * page_size + offset
 *               (as ftd_build_tables makes them); negative: the token's keys and values go
 *               nowhere.  v is needed, k_out and v_out are NULL.  Two tokens of one call must
 *               not name one slot.
 *   k_cache, v_cache, scales : as in ftd_decode_mha / _paged (NULL: the pool).  Rows are
 *               rounded once from fp32 to the cache type; INT8 rows are codes and a scale
 *               as ftd_decode_mha appends them.  Only the named rows are written.
 * A slot past the cache's end writes nothing and raises FTD_ERR_BAD_PAGE.  Every row is the one
 * that the step would append, where qkv and cache type are one.  Launches one kernel.
 */
ftd_status ftd_norm_rope_qkv(ftd_ctx* ctx, const void* q, const void* k, const void* v, int64_t q_stride, int64_t kv_stride,
                             const void* qkv_bias, const void* q_weight, const void* k_weight, float eps, float weight_offset,
                             const int32_t* positions, int64_t n_tokens, void* q_out, void* k_out, void* v_out,
                             const int32_t* slots, void* k_cache, void* v_cache, float* scales, void* stream);

/*
 * ftd_build_tables -- block tables and slot maps from request lengths: brings every slot
 * from old_lens[b] to new_lens[b] cached rows (negative: inactive, no rows), by the pages
 * of a free list, and says where the rows between go.
 *   old_lens, new_lens : device int32 [B].  A slot grows, shrinks (an eviction, rejected
 *               tokens), begins (old <= 0) or ends (new <= 0).
 *   served    : device int32 [B], may be either list: new_lens[b], or old_lens[b] where the
 *               slot was not served: a length above Lmax (FTD_ERR_SEQ_OVERFLOW), or too few
 *               pages left.  The latter is no error; the slot keeps its pages and can ask
 *               again.  Slots are served in order: once one has to wait, so do all later
 *               ones that ask for pages.
 *   block_table : device int32 [B][ceil(Lmax / page_size)]: the first ceil(old_lens[b] /
 *               page_size) entries of a slot are its pages; entries for its new rows are
 *               written, no others.
 *   free_pages, n_free : device int32 [num_pages] and [1]: a stack, its top at n_free - 1.
 *               Entries that slots give back are pushed in (slot, entry) order, then those
 *               asked for are popped in that order, so pages given back are used again first.
 *               Pages have no counts of users: one that two slots' tables hold comes back twice,
 *               and a shared prefix's pages belong to a slot of their own that outlives the others.
 *   n_free_out : device int32 [1], NULL or n_free: in place.
 *   offsets   : device int32 [B + 1] or NULL: new tokens of the slots before b, packed.
 *   slots     : device int32 [max_tokens] or NULL: for each new token, in packed order, its
 *               place in the cache as ftd_norm_rope_qkv takes it; -1 from offsets[B] on.
 *   positions : device int32 [max_tokens] or NULL: its position; 0 from offsets[B] on.
 *               More than max_tokens new tokens raise FTD_ERR_SEQ_OVERFLOW, and those past
 *               it are left out of both lists.  max_tokens 0: as with both lists NULL.
 * On a contiguous context block_table, free_pages, n_free and n_free_out are NULL.  A page
 * outside [0, num_pages) that changes hands or holds a new token raises FTD_ERR_BAD_PAGE (its
 * tokens get -1), and so do an n_free outside [0, num_pages] and pages given back that the
 * list has no room for.  Other overlaps of outputs are refused.  Launches one kernel, whose
 * result does not depend on the order of anything.
 */
ftd_status ftd_build_tables(ftd_ctx* ctx, const int32_t* old_lens, const int32_t* new_lens, int32_t* served, int32_t* block_table,
                            int32_t* free_pages, const int32_t* n_free, int32_t* n_free_out, int32_t* offsets, int32_t* slots,
                            int32_t* positions, int64_t max_tokens, void* stream);

/*
 * ftd_enable_scores -- allocate the workspace of ftd_decode_mha_scored and
 * ftd_cache_evict: 4 bytes per (query row, cache position) of the context, 4 more
 * per (kv head, position) and some constants.  One cudaMalloc, freed by
 * ftd_destroy; clearing runs on `stream`.  A second call does nothing.
 */
ftd_status ftd_enable_scores(ftd_ctx* ctx, void* stream);

/*
 * ftd_decode_mha_scored -- the step of ftd_decode_mha (of ftd_decode_mha_paged on a
 * paged context), which also adds each position's attention weight to a plane:
 *   acc_out[b][h][t] = (t < L_b ? acc[b][h][t] : 0) + sum of p_t over the T * Hq / Hkv
 *   query rows of kv head h, for t = 0 .. L_b + T - 1,
 * in fp32 and in a fixed order.  A row whose window or causal limit hides t adds
 * nothing there.  With T > 1 every token's row counts, also of tokens that the
 * caller then rejects.
 *   block_table : as in ftd_decode_mha_paged; NULL on a contiguous context.  With a window and acc_out
 *               apart from acc, the weights behind the window are copied, so entries there
 *               name the slot's own pages too, or none: outside [0, num_pages) they are passed over.
 *   acc       : device fp32 plane laid out like one INT8 scale plane: [B][Hkv][Lmax],
 *               paged [num_pages][Hkv][page_size]; 16-byte aligned.
 *   acc_out   : the same, NULL or acc: in place.  Entries past L_b + T - 1, and
 *               slots without work, keep what they hold.
 *   positions : device int32 plane of the same layout, or NULL: the new rows' entries
 *               become next_pos[b] + j (every kv head's).  Older entries are kept.  Apart
 *               from acc and acc_out.
 *   next_pos  : device int32 [B], the sequence position of the slot's first new token
 *               (L_b as long as nothing was evicted); needed with positions.
 * Pages that two active slots share would take both slots' weights in no order: a
 * page belongs to one slot here.
 * A slot with a bad entry among its visible pages (FTD_ERR_BAD_PAGE) keeps its acc_out and
 * positions entries, and so do all slots of a call that gives up on a copy, and of later ones
 * until ftd_get_error has reported that FTD_ERR_DEVICE_TIMEOUT: the weights gathered before
 * are not lost, and the call can be made again.
 * Other arguments, out and the sticky errors as in ftd_decode_mha, and so are the
 * appended rows, but for an INT8 row's scale: absmax * (1 / 127) in fp32 here, at most an
 * ulp from ftd_decode_mha's absmax / 127 (codes are round(k' / scale) in both, so one that
 * lies on a rounding border can differ by 1).  Launches two kernels.
 */
ftd_status ftd_decode_mha_scored(ftd_ctx* ctx, const void* q, const void* k_new, const void* v_new,
                                 const void* qkv_bias, void* k_cache, void* v_cache, const int32_t* block_table,
                                 const int32_t* seq_lens, float* scales, const int32_t* next_pos, const float* acc,
                                 float* acc_out, int32_t* positions, void* out, void* stream);

/*
 * ftd_cache_evict -- bring every slot with more than `budget` cached rows down to
 * budget, each kv head by its own weights.  Of its L_b = seq_lens[b] rows a head keeps
 *   first those whose position is below `sinks` (negative ones too) or at least
 *   next_pos[b] - `recent` (later ones too, whatever `recent` is),
 *   then the largest acc (NaN below all), equal ones (0 and -0 are) by the lower row.
 * Rows are not kept in order: the j-th kept row at index >= budget moves into the
 * j-th row below budget that is not kept, K and V (INT8: and their scales), weight
 * and position; no other row moves, and rows from budget on keep their old content.
 * Attention does not depend on the order (positions are in K), so ftd_decode_mha runs
 * on from new_lens; on a paged context the pages past them are free to reuse.
 *   k_cache, v_cache, scales, block_table : as in ftd_decode_mha / _paged (NULL caches
 *               and scales: the pool).
 *   acc, positions : planes as in ftd_decode_mha_scored, 4-byte aligned.
 *   acc_out, positions_out : planes that take the kept rows' entries 0 .. new length - 1;
 *               NULL or the input plane: in place.  Other overlaps are refused.
 *   new_lens  : device int32 [B], may be seq_lens: budget, or L_b where that is no more.
 * A page that holds rows of a slot over the budget must be that slot's alone.
 * Inactive slots (L_b < 0) are left alone; L_b > Lmax raises FTD_ERR_SEQ_OVERFLOW, a
 * bad table entry FTD_ERR_BAD_PAGE (that slot's rows stay where they are, its length
 * and planes are undefined).  Needs 1 <= budget <= Lmax and recent + sinks <= budget, a
 * context without a window, and Lmax up to 2^30 (UNSUPPORTED above).  Launches two kernels.
 */
ftd_status ftd_cache_evict(ftd_ctx* ctx, void* k_cache, void* v_cache, float* scales, const int32_t* block_table,
                           const int32_t* seq_lens, const int32_t* next_pos, const float* acc, float* acc_out,
                           const int32_t* positions, int32_t* positions_out, int32_t* new_lens, int budget,
                           int recent, int sinks, void* stream);

/*
 * ftd_cross_mha -- cross attention of the T = q_len tokens (or beams) of every slot to
 * an encoder's states, kept as K and V rows in the layout of a cache:
 *   out[b][j][h] = softmax(scale * (q[b][j][h] + q_bias[h]) . K_mem[b][h'][0 .. M_b - 1]) V_mem,
 * M_b = mem_lens[b], h' the kv head of h.  Nothing is appended, every token sees the
 * whole memory, and the tokens of a slot share one pass over it.
 *   q        : device [B][T][Hq][D], out [B][T][Hq][D] of out_dtype.
 *   q_bias   : device [Hq * D] or NULL.
 *   k_mem, v_mem : device [B][Hkv][Lmax][D] of the cache dtype, read only (INT8: with
 *              scales [2][B][Hkv][Lmax]); NULL: the context's pool.  Rows from M_b on
 *              may hold anything.
 *   mem_lens : device int32 [B].  M_b <= 0 gives zeros; M_b > Lmax gives zeros and
 *              raises FTD_ERR_SEQ_OVERFLOW.
 * Runs on any context without pages and without a window.  Launches one kernel.
 */
ftd_status ftd_cross_mha(ftd_ctx* ctx, const void* q, const void* q_bias, const void* k_mem, const void* v_mem,
                         const int32_t* mem_lens, const float* scales, void* out, void* stream);

/*
 * ftd_enable_prefix -- allocate the workspace of ftd_decode_mha_prefix: for each SM and for each
 * kv head and block of query rows a partial result over the prefix; for the slots' own rows
 * either an fp32 copy of out and two numbers per query row, or, where the prefix's kernel takes
 * them too, two partial results per SM and one per slot and kv head.  One cudaMalloc, freed by ftd_destroy; nothing is launched, so
 * the stream is not used.  A second call does nothing.  UNSUPPORTED
 * above 32768 query rows per kv head (B * T * Hq / Hkv), INVALID_ARG with a window.
 */
ftd_status ftd_enable_prefix(ftd_ctx* ctx, void* stream);

/*
 * ftd_decode_mha_prefix -- the step of ftd_decode_mha (of ftd_decode_mha_paged on a paged
 * context) for slots that share a long prefix, as the samples of one question or the chats
 * behind one system prompt do: slot b's tokens attend to the first prefix_lens[b] rows
 * of the prefix and to the slot's own rows, those of its cache and the new ones,
 *   out[b][j][h] = softmax over both of scale * q'[b][j][h] . K, times V.
 * The prefix is read once for all slots: with B slots its products are matrix products
 * with B * T * Hq / Hkv rows, on the tensor cores for fp16, bf16 and INT8 caches.
 * It pays from about B * prefix_rows * Hkv = 500000 rows of 128 (8 slots behind 8192 rows with 8 kv heads, 4 with 32; INT8
 * as much with 8 kv heads and two to eight times that with 32; multi-query caches always with up to 8 slots): below, ftd_decode_mha_paged over block tables that name the
 * prefix's pages in every slot is as fast or faster.  Here / there, us: 32 kv heads, fp16, behind 768 rows 4 / 16 / 64 slots
 * 42 / 47 / 66 against 25 / 50 / 150, behind 8192 rows 2 / 4 / 16 slots 61 / 66 / 73 against 58 / 93 / 320; 64 on 8 heads, bf16, behind 2048 rows 16 / 32 slots
 * 46 / 50 against 40 / 62, behind 32768 rows 2 / 4 / 64 slots 62 / 62 / 128 against 60 / 89 / 1092.
 *   k_prefix, v_prefix : device [Hkv][prefix_rows][D] of the cache dtype, 16-byte aligned, read
 *               only, apart from the caches and out; INT8 with prefix_scales, device fp32 [2][Hkv][prefix_rows].  On a
 *               paged context NULL: the prefix lies in pages of the pool, and
 *   prefix_table : device int32 [ceil(prefix_rows / page_size)] names them (NULL on a
 *               contiguous context).  No slot's block table may have them in reach of a
 *               new row.
 *   prefix_rows : rows of the prefix, >= 0; 0: ftd_decode_mha's call.  Refused where prefix_rows * Hkv, or ceil(prefix_rows / 64)
 *               times the blocks of 64 to 256 query rows of a kv head, passes 31 bits.
 *   prefix_lens : device int32 [B].  A slot that shares nothing has 0 (or less); one above
 *               prefix_rows sees prefix_rows and raises FTD_ERR_SEQ_OVERFLOW.
 * seq_lens counts the slot's own rows: 0 as long as it has only the prefix.  Keys carry their
 * positions already, so the slot's own rows start wherever the caller turned them to.
 * Rows of the prefix from the longest prefix_lens on may hold anything; rows that some slot
 * sees hold finite values.
 * Other arguments, out, the appended rows (with prefix_rows above 0 an INT8 row's scale as in ftd_decode_mha_scored) and
 * the sticky errors as in ftd_decode_mha; a page of the prefix outside [0, num_pages) raises
 * FTD_ERR_BAD_PAGE, and what the slots see of it is undefined.
 * fp16 and bf16 caches: the tensor cores take the weights as pairs of numbers of that type (about 16 mantissa bits with
 * bf16, 22 with fp16), as ftd_decode_mha does, and q as it is where it is of the cache's type and has no bias, else as a pair
 * too.  INT8 caches: codes are exact, scales multiply scores and weights in fp32; the weights are pairs of bf16 numbers, q one
 * fp16 or bf16 number where it is of that type and has no bias, else such a pair too.  Launches two or
 * three kernels: the slots' own rows are taken beside the prefix or by the step's kernel.
 */
ftd_status ftd_decode_mha_prefix(ftd_ctx* ctx, const void* q, const void* k_new, const void* v_new, const void* qkv_bias,
                                 void* k_cache, void* v_cache, const int32_t* block_table, const int32_t* seq_lens,
                                 float* scales, const void* k_prefix, const void* v_prefix, const float* prefix_scales,
                                 const int32_t* prefix_table, int64_t prefix_rows, const int32_t* prefix_lens, void* out,
                                 void* stream);

/* Size of the fixed device array that ftd_decode_mha_noalloc uses as scratch. */
#define FTD_NOALLOC_SCRATCH_BYTES (8u << 20)

/*
 * ftd_decode_mha_noalloc -- the decode step of ftd_decode_mha for callers that
 * must not allocate device memory.  The pages describe nothing like it: it
 * exists for callers that cannot call cudaMalloc at all -- a plugin inside a
 * host runtime whose own allocator owns all device memory, or a serving loop
 * that forbids allocation (which can synchronise the device or fail) after
 * start-up -- and so cannot create a context with ftd_init.
 *
 *   cfg              : shape, dtypes and options, same rules as ftd_init,
 *                      except that page_size must be 0 (contiguous caches).
 *   q ... out        : as in ftd_decode_mha, all caller-owned device memory;
 *                      k_cache and v_cache are required (there is no pool), and
 *                      so are scales for an INT8 cache.
 *   device_err       : device uint32, or NULL.  When given, the kernel ORs its
 *                      error bits into it (1 = some seq_lens[b] + q_len > max_len,
 *                      2 = a bounded wait gave up); the caller reads and clears
 *                      it.  When NULL those bits are dropped (overflowing slots
 *                      still get a zero output).
 *   stream           : cudaStream_t as void*.
 *
 * It allocates nothing: no cudaMalloc, cudaFree or allocating library call.
 * It runs the kernel ftd_decode_mha would run for the same config; for the
 * tensor-core kernel it encodes the caches' tensor maps on the host at every
 * call (a context caches them), so its results are ftd_decode_mha's bytes.
 * Its split-K partials, counters and error word live in one static device
 * array of FTD_NOALLOC_SCRATCH_BYTES (8 MiB) that every GPU loading the
 * library holds until the process exits.  A configuration that needs more is
 * rejected with FTD_ERR_INVALID_ARG, and ftd_last_error() gives the bytes it
 * needs.  The need is one partial slot per segment (max_batch * n_kv_heads *
 * query-row blocks per kv head) plus, per SM, one slot per worker: the CUDA-core
 * kernel's warps per block (8, or 12 for INT8 caches with blocks of at most 2
 * query rows), or 1 for the tensor-core kernel; a slot holds (2 + head_dim)
 * floats per query row of a block, plus counters and the error word.
 * The first call on each device does a one-time set-up with that device
 * current (it looks up the array's device address and raises the kernel's
 * shared-memory limit); make that first call before any stream capture.
 * Every call clears the counters and error word it uses at the start, on
 * `stream`.  All calls share the one array: calls whose kernels overlap in
 * time on the same GPU race and give wrong results, so issue them on one
 * stream or order them with events.
 */
ftd_status ftd_decode_mha_noalloc(const ftd_config* cfg, const void* q, const void* k_new,
                                  const void* v_new, const void* qkv_bias, void* k_cache,
                                  void* v_cache, const int32_t* seq_lens, float* scales, void* out,
                                  uint32_t* device_err, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FTD_H */
