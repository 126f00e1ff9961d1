/*
 * hg.h - C ABI of the vocab-parallel LM-head logits gather on a two-parity
 * Lamport mailbox, for TP virtual ranks on one GPU.
 *
 * The operation (vLLM API page
 * "vllm.models.kimi_k3.nvidia.specialized_decode.runtime.logits_gather",
 * module docstring and class HeadGather): each of TP ranks holds an [M, W]
 * BF16 logits shard (W = V / TP vocab columns). Seen as 32-bit words, rank r's
 * row m is stored into the same row of each rank's mailbox (the pushing rank's
 * own included), starting at word column r * W / 2: NCCL's all-gather order. A mailbox word
 * that has not arrived holds the sentinel, the BF16 pair (+0, -0) = 0x80000000
 * (low half +0, high half -0); a data word equal to the sentinel is sent as
 * (+0, +0) = 0x00000000, every other word moves unchanged. Each rank polls its
 * mailbox row until no sentinel word is left, copies the row to its [M, V]
 * output and writes the sentinel back (re-arms). Two mailbox parities
 * alternate per call, so that a push never lands in a row that the previous
 * call may still be reading.
 *
 * On one GPU the TP ranks are virtual: every rank has its own shard, mailbox
 * and output allocation on the same device, and one kernel launch runs all of
 * them.
 *
 * Conventions for every entry point:
 *  - Return value: HG_OK (0) or one of the HG_ERR_* codes below.
 *  - "device pointer": memory of the device that was current at hg_create;
 *    the caller keeps that device current for every later call. A gather or
 *    hg_rearm with another one current answers HG_ERR_ARG.
 *  - Calls on one handle are not thread-safe; every gather of a handle runs on
 *    one stream, in call order (the class docstring's one-stream assumption).
 *  - A call that returns an error other than HG_ERR_TIMEOUT changed nothing:
 *    neither the parity nor any mailbox nor any output.
 */
#ifndef HG_H_
#define HG_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t; NULL is the legacy default stream. */
typedef struct CUstream_st *hg_stream_t;

/* Opaque, library-owned state of one gather: the mailboxes, the parity, the
 * device status word and the launch shapes. */
typedef struct hg_handle hg_handle;

enum {
  HG_OK = 0,
  HG_ERR_ARG = 1,      /* invalid argument: NULL, misaligned, out of range */
  HG_ERR_ROWS = 2,     /* row count M not served by this handle (where
                          HeadGather.__call__ falls back to the stock gather) */
  HG_ERR_CAPTURE = 3,  /* stream is capturing a CUDA graph (HeadGather also
                          falls back to the stock gather under capture) */
  HG_ERR_CUDA = 4,     /* a CUDA runtime call failed (allocation, launch) */
  HG_ERR_TIMEOUT = 5,  /* a poll gave up: some pushed word never arrived */
  HG_ERR_STATE = 6     /* the handle holds an unrecovered device error;
                          call hg_rearm before gathering again */
};

/* Largest TP supported by one handle. */
#define HG_MAX_TP 32

/* Optional settings of hg_create_ex. Zero in any field selects the default. */
typedef struct hg_options {
  uint64_t poll_timeout_ns; /* bound of every poll; default 1e9 (1 s) */
  int elems_per_lane;       /* 16-byte vectors (or words) per lane per unit:
                               1 to 6 for tp <= 16, 1 or 2 above; default
                               chosen per row count */
  int ctas;                 /* CTAs of the gather kernel (32 * tp threads each);
                               default chosen per row count; clamped to what is
                               co-resident. Also caps the grid of
                               hg_gather_fused (default one CTA per SM) */
  int prefetch;             /* 0: chosen per row count (off unless tuned), 1: the
                               next push's shard loads are issued one iteration
                               ahead of its stores (overlapping a poll), 2: off */
  int cooperative;          /* 0 (default): programmatic dependent launch, the
                               next call's launch overlaps this one; 1:
                               cooperative launch, the runtime itself checks
                               that every CTA is co-resident (no overlap) */
  int device_parity;        /* 0 (default): the host keeps the parity and calls
                               on a capturing stream are refused
                               (HG_ERR_CAPTURE); 1: the parity lives in device
                               memory, each call's kernel reads it and flips it
                               once every CTA has read it, so calls may be
                               captured into a CUDA graph and replayed; the
                               host learns the parity only at hg_sync */
  int autotune;             /* 0 (default): launch shapes from a fixed rule; 1:
                               hg_create_ex times candidate shapes (elements
                               per lane, CTAs, prefetch) of hg_gather for every
                               served row count on the device and keeps the
                               fastest (hg_gather_stats keeps the fixed rule)
                               (the fixed rule's shape unless another is
                               faster by at least 3 %, in the sweep and again
                               head to head). The
                               candidates honour the fields above that are
                               set. The timed calls rotate over inputs and
                               outputs in a zero-filled pool of max(256 MB,
                               tp * M * (W + tp * W) * 2 bytes) that is freed
                               before returning; row counts above 16, and those
                               whose one set would exceed 1 GB, keep the fixed
                               rule. It costs
                               tens of milliseconds per served row count at the
                               decode sizes and changes no result, only speed */
  int timeline_calls;       /* 0 (default): off; n > 0: a measurement build of
                               the gather records, for each of the last n
                               calls of hg_gather, hg_gather_stats and
                               hg_gather_fused, per CTA when it started, when
                               its wait for the previous kernel returned and
                               when each warp finished (hg_timeline). Needs shard_cols % 8 == 0,
                               tp <= 16 and no prefetch; it costs a few stores
                               per CTA and changes no result */
} hg_options;

/*
 * hg_create - allocate and arm the mailboxes of one gather
 * (HeadGather.__init__: LamportRows(group, device, (2, cap, words * tp),
 * PAIR_SENT), parity = 0, device synchronised before returning).
 *
 *   tp          virtual ranks, 1 <= tp <= HG_MAX_TP
 *   shard_cols  W, BF16 columns per rank; even (W % 8 == 0 selects the 16-byte
 *               vector path, other even W a 4-byte word path)
 *   cap         mailbox rows per parity, >= max(rows)
 *   rows        the served row counts, each in [1, cap] (HeadGather's `rows`);
 *               NULL with nrows == 0 serves every M in [1, cap]
 *   out         receives the handle
 *
 * Allocates, on the current device, tp mailboxes of 2 * cap * tp * W BF16
 * each (parity-major, then row, then column) plus a status word, fills every
 * mailbox word with 0x80000000 and synchronises the device. The handle owns
 * that memory until hg_destroy. Errors: HG_ERR_ARG (bad sizes, rows out of
 * range, size overflow), HG_ERR_CUDA (no device, allocation failure).
 */
int hg_create(int tp, int shard_cols, int cap, const int *rows, int nrows, hg_handle **out);

/* hg_create with settings; opt may be NULL. Same contract as hg_create. */
int hg_create_ex(int tp, int shard_cols, int cap, const int *rows, int nrows,
                 const hg_options *opt, hg_handle **out);

/* Free the mailboxes and the handle; waits for the device first. NULL is a
 * no-op. Always returns HG_OK unless freeing fails (HG_ERR_CUDA).
 * The pages have no counterpart: HeadGather's mailbox lives as long as the
 * model that installed it. */
int hg_destroy(hg_handle *h);

/*
 * hg_gather - one gather call (HeadGather.__call__ and the kernel of the module
 * docstring): push, poll, copy, re-arm, for every virtual rank, in one
 * persistent kernel launch on `stream`. Asynchronous.
 *
 *   shard_ptrs  tp device pointers; shard_ptrs[r] is rank r's [M, W] BF16
 *               shard, row-major, rows contiguous (row stride W); 16-byte
 *               aligned on the vector path, 4-byte aligned otherwise; read only
 *   out_ptrs    tp device pointers; out_ptrs[d] is rank d's [M, tp * W] BF16
 *               output, row-major, fully overwritten; same alignment rule; must
 *               not overlap a shard or another output
 *   M           rows this call; must be a served row count
 *   stream      the stream every gather of this handle runs on
 *
 * Uses parity hg_parity(h), then flips it. The caller owns the shards and the
 * outputs; the library owns the mailboxes.
 *
 * The launch may start while the previous kernel on `stream` still runs (a
 * programmatic dependent launch). Before it waits for that kernel to
 * complete, each CTA asks L2 to prefetch the first bytes of shard it will
 * read (on the vector path). That is a cache hint only: every value the
 * gather reads is read after the previous kernel has completed, so the
 * shards may be that kernel's output.
 *
 * Co-residency: the kernel's CTAs wait on one another's pushes, so its whole
 * grid must become resident. The grid is sized for an otherwise idle GPU.
 * Kernels running concurrently on other streams can hold SM resources and
 * keep part of the grid from starting until they release them; the call is
 * delayed that long, and if that exceeds the poll bound (for example a
 * persistent kernel on another stream, including another gather: two gathers
 * on different streams can each hold the slots the other needs) it reports
 * HG_ERR_TIMEOUT at hg_sync.
 * Issue such work on the same stream, or create the handle with
 * hg_options.cooperative = 1, where the runtime itself guarantees
 * co-residency (at the cost of the launch overlap). Errors, all before any device work
 * and with no parity flip: HG_ERR_ARG (NULL handle or pointer, misaligned
 * pointer), HG_ERR_ROWS (M not served), HG_ERR_CAPTURE (stream capturing,
 * unless the handle has device_parity), HG_ERR_CUDA (launch failed; parity
 * not flipped). A poll that times out on the
 * device is reported by the next hg_sync; until hg_rearm every later gather
 * of the handle does no device work.
 */
int hg_gather(hg_handle *h, const void *const *shard_ptrs, void *const *out_ptrs, int M,
              hg_stream_t stream);

/*
 * hg_gather_host - hg_gather whose shards and outputs may live in page-locked
 * host memory (cudaHostAlloc, cudaMallocHost or cudaHostRegister), as well as
 * in device memory of the handle's device. The pages define the gather on
 * device buffers only; this entry point is this library's end-to-end form for
 * a host that holds the logits: the same kernel reads the shards from host
 * memory and writes the outputs into host memory directly over the
 * host-device link (no staging copies), while the mailboxes stay in device
 * memory. Same arguments, contract and errors as hg_gather, plus:
 *
 *   no L2 prefetch of the shards before the wait (the host may still be
 *   writing them);
 *   every pointer is checked with cudaPointerGetAttributes and replaced by its
 *   device-side address; pageable host memory, memory of another device and
 *   unknown addresses give HG_ERR_ARG before any device work.
 *
 * The outputs are complete in host memory once the stream has passed the
 * call (e.g. after hg_sync or a stream synchronisation).
 */
int hg_gather_host(hg_handle *h, const void *const *shard_ptrs, void *const *out_ptrs, int M,
                   hg_stream_t stream);

/* Wait for `stream`, then read the device status word. Returns HG_OK,
 * HG_ERR_TIMEOUT (a poll gave up; mailbox contents undefined until hg_rearm)
 * or HG_ERR_CUDA. Failure detection of this library; the pages have no
 * counterpart (their polls are unbounded). */
int hg_sync(hg_handle *h, hg_stream_t stream);

/* Recovery after an error: refill every mailbox word of both parities with
 * the sentinel, re-arm the statistics cells and the fused producer's split
 * cells, clear the status words and set the parity to 0 (host and device
 * copies), on `stream`, asynchronously. It restores the state that
 * HeadGather.__init__ leaves (mailboxes armed with PAIR_SENT, parity 0);
 * recovery itself has no counterpart on the pages. */
int hg_rearm(hg_handle *h, hg_stream_t stream);

/* Parity the next hg_gather uses (0 or 1; starts at 0, flips per served call
 * as `self.parity ^= 1` in HeadGather.__call__), or -1 for NULL. With
 * device_parity, the parity as of the last hg_sync or hg_rearm. */
int hg_parity(const hg_handle *h);

/* Rank `rank`'s mailbox for inspection: device pointer to [2][cap][tp * W]
 * BF16 (parity-major) and its size in bytes. Owned by the handle; read it only
 * while no gather is in flight. Errors: HG_ERR_ARG. Test surface: the layout
 * is that of LamportRows(group, device, (2, cap, words * tp), PAIR_SENT) in
 * HeadGather.__init__, but the pages expose no accessor. */
int hg_mailbox(const hg_handle *h, int rank, const void **dev_ptr, size_t *bytes);

/* Launch shape that hg_gather uses for row count M: CTAs, threads per CTA,
 * elements per lane and whether the next push's shard loads are issued one
 * iteration ahead (1) or not (0). Any output pointer may be NULL. Errors:
 * HG_ERR_ARG, HG_ERR_ROWS. Inspection only; the pages' counterpart,
 * gather_ctas(m, ...) in HeadGather.__init__, is named but not printed. */
int hg_launch_shape(const hg_handle *h, int M, int *ctas, int *threads, int *elems_per_lane,
                    int *prefetch);

/* One CTA's record in the timeline of hg_options.timeline_calls: %globaltimer
 * nanoseconds at entry (before the kernel waits for the previous kernel on
 * the stream), once that wait returned, and when warp d finished (d < tp;
 * warps of CTAs that gave up record nothing); for tp <= 14, warp_done[14]
 * holds instead the index of the SM the CTA ran on. In hg_gather_stats calls with
 * tp < 16, warp_done[15] holds when warp 0 finished its share of the gather
 * and turned to reducing the statistics of its rows, and for tp <= 8 warp 0
 * also records in warp_done[8..12]: its first poll complete, its first
 * outputs stored, its first unit folded, and (CTAs g < M, reducing row g) all
 * of row g's cells arrived and folded, and row g's statistics written. hg_gather_fused calls
 * (one CTA per SM; recorded when the handle's grid records have room for it)
 * use the same slots differently: entry; set-up done (tensor memory and
 * barriers ready); warp_done[i] (i < 8): the epilogue has pushed its item i;
 * warp_done[8 + j] (j < 6): it has consumed the neighbour CTA's item j inside
 * its loop; warp_done[14]: the epilogue loop is done; warp_done[15]: the CTA
 * is done. */
#define HG_TIMELINE_SLOTS 18
typedef struct hg_timeline_record {
  uint64_t entry;
  uint64_t waited;
  uint64_t warp_done[HG_TIMELINE_SLOTS - 2];
} hg_timeline_record;

/*
 * hg_timeline - the timeline of a handle created with timeline_calls = n:
 * device pointer to [n][ctas] hg_timeline_record (ctas = the largest grid of
 * any served row count; a call of a smaller grid fills its first CTAs), and
 * the index of the record the next call writes (calls fill records 0, 1, ...
 * in call order and wrap around after n). Read it only while no gather of the
 * handle is in flight. A measurement surface with no counterpart on the
 * pages. Errors: HG_ERR_ARG (NULL, or a handle without a timeline).
 */
int hg_timeline(const hg_handle *h, const hg_timeline_record **dev_ptr, int *calls, int *ctas,
                int *next);

/*
 * hg_probe - measurement kernels that bound the gather's latency from below;
 * no counterpart on the pages. Both are launched as the gather is (a
 * programmatic dependent launch of `ctas` CTAs of `threads` threads, a
 * multiple of 32, at most 512) on `stream`:
 *
 *   kind 0  empty: wait for the previous kernel, let the next one launch,
 *           return. The cost of one dependent launch of that grid.
 *   kind 1  handoff: warp w of CTA g stores one 16-byte vector per lane into
 *           its slot, lets the next kernel launch, polls the slot of CTA
 *           g + 1 (mod ctas) until it arrives (relaxed loads, bounded by 1 s),
 *           stores it to an output and re-arms that slot: the gather's push,
 *           poll, copy and re-arm for one vector per lane and no shard read.
 *
 *   scratch  device buffer of hg_probe_scratch_bytes(ctas, threads) bytes,
 *            16-byte aligned, owned by the caller; kind 1 needs it armed by
 *            kind 2 (fill the slots with the sentinel, clear the status word)
 *            once before its first launch, and leaves it armed; the status
 *            word (the last 4 bytes) becomes 1 if a poll gave up.
 *
 * Errors: HG_ERR_ARG (kind, sizes, NULL or misaligned scratch), HG_ERR_CUDA.
 */
int hg_probe(int kind, int ctas, int threads, void *scratch, hg_stream_t stream);

/* Bytes of the scratch buffer of hg_probe for that grid. */
size_t hg_probe_scratch_bytes(int ctas, int threads);

/*
 * Test hook for failure detection: make rank `rank`'s push skip its rows in
 * every later gather, plain, with statistics or fused (the fused producer
 * still computes and optionally stores that rank's logits) (rank = -1 turns
 * it off). The pollers of the other ranks
 * then wait for words that never arrive and give up after the poll bound;
 * hg_sync reports HG_ERR_TIMEOUT. No device fault, trap or endless wait is
 * involved. Errors: HG_ERR_ARG. No counterpart on the pages.
 */
int hg_debug_skip_push(hg_handle *h, int rank);

/*
 * hg_gather_fused - the vocab-parallel LM head and the gather in one kernel
 * (API page, module docstring: the lm_head's [M, V / TP] logits per rank, then
 * the gather). For every rank r:
 *   logits_r[m][n] = bf16_rn(sum_k hidden_r[m][k] * weight_r[n][k])
 * with fp32 accumulation on the tensor cores; the GEMM's epilogue pushes the
 * bf16 words straight into every rank's mailbox (sentinel rewrite included),
 * and the same launch polls, copies to out_ptrs and re-arms, exactly as
 * hg_gather does on those logits. Asynchronous on `stream`; uses parity
 * hg_parity(h), then flips it.
 *
 *   hidden_ptrs  tp device pointers to [M, K] bf16, row-major, 16-byte aligned
 *   weight_ptrs  tp device pointers to [W, K] bf16 (nn.Linear layout: vocab
 *                rows, hidden columns), row-major, 16-byte aligned
 *   logits_ptrs  NULL, or tp device pointers (each may be NULL) that receive
 *                rank r's bf16 logits [M, W] as computed (before the rewrite)
 *   out_ptrs     tp device pointers to [M, tp * W] bf16, as for hg_gather
 *   M            rows: served by the handle and <= 16
 *   K            hidden size: a positive multiple of 64
 *
 * Requires tp <= 16 and W a multiple of 128. One CTA per SM (a cooperative
 * launch; hg_options.ctas caps the grid). When the vocab tiles do not divide
 * evenly over the CTAs, the last tiles are split along K over several CTAs,
 * whose fp32 partials meet in the handle's split cells; the sum of the parts
 * may round differently from one accumulation over K (fp32), which the
 * logits tolerance covers, and the gathered outputs are always exactly the
 * gather of the returned logits. Errors, before any device work and with no
 * parity flip: HG_ERR_ARG, HG_ERR_ROWS, HG_ERR_CAPTURE, HG_ERR_STATE,
 * HG_ERR_CUDA (launch or tensor-map encoding failed). A wait that times out is
 * reported by hg_sync, as for hg_gather; hg_rearm also re-arms the split
 * cells.
 */
int hg_gather_fused(hg_handle *h, const void *const *hidden_ptrs, const void *const *weight_ptrs,
                    void *const *logits_ptrs, void *const *out_ptrs, int M, int K,
                    hg_stream_t stream);

/*
 * hg_stock_gather - the baseline without a mailbox: the rank-order concat of
 * NCCL's all-gather (the page's stock LogitsProcessor gather: all-gather into
 * [TP, M, V / TP], then a copy to [M, V]) done as tp * tp cudaMemcpy2DAsync
 * copies on `stream`. Moves every word unchanged (no sentinel rewrite).
 * Pointers and layouts as in hg_gather (no alignment rule beyond 2 bytes).
 * Errors: HG_ERR_ARG, HG_ERR_CUDA.
 */
int hg_stock_gather(int tp, int shard_cols, const void *const *shard_ptrs,
                    void *const *out_ptrs, int M, hg_stream_t stream);

/* Largest mailbox that one hg_gather_static call may use, in bytes:
 * tp * M * tp * shard_cols * 2 (every rank's [M, V] BF16 rows, one parity).
 * At TP8, V=163840 (shard_cols 20480) that is up to M = 9 rows. */
#define HG_STATIC_MAILBOX_BYTES (24u * 1024u * 1024u)

/*
 * hg_gather_static - hg_gather for callers that cannot allocate device memory.
 * The pages have no counterpart to this entry point: their gather always owns a
 * mailbox allocated at construction.
 *
 * Some callers cannot call cudaMalloc: a serving engine whose caching
 * allocator has already reserved the GPU's free memory, a plug-in inside a
 * host framework that forbids allocations outside its own allocator, or a
 * latency-critical loop that cannot pay for cudaMalloc/cudaFree's implicit
 * device synchronisation. This call allocates nothing. Its mailbox and status
 * words live in a fixed __device__ array inside the library
 * (HG_STATIC_MAILBOX_BYTES + 256 bytes), which every GPU that loads the
 * library holds until the process exits.
 *
 *   tp, shard_cols  as for hg_create (1 <= tp <= HG_MAX_TP, shard_cols even)
 *   shard_ptrs      tp device pointers to [M, shard_cols] BF16, as for hg_gather
 *   out_ptrs        tp device pointers to [M, tp * shard_cols] BF16, as for
 *                   hg_gather
 *   M               rows, >= 1, with tp * M * tp * shard_cols * 2 <=
 *                   HG_STATIC_MAILBOX_BYTES
 *   status_out      optional device pointer to one int32 that receives, in
 *                   stream order, 0 on success or 1 if a poll gave up; NULL: not
 *                   reported
 *   stream          the stream of the call
 *
 * Same result as hg_gather on the same shards. The call works on the device
 * that is current when it is made: `stream` and every pointer must belong to
 * that device (a stream of another device gives HG_ERR_ARG). The first call
 * on a device looks up the array's device address (cudaGetSymbolAddress, with
 * that device current), so make that first call before any stream capture. Every call
 * shares the array and finds it as the previous call left it: each call clears
 * the status words and re-arms its mailbox region before gathering, on
 * `stream`. Calls whose device work overlaps (other streams or threads) race on
 * the array. No parity state is kept. Errors, before any device work:
 * HG_ERR_ARG (bad sizes, NULL or misaligned pointers, a mailbox larger than
 * HG_STATIC_MAILBOX_BYTES, or a stream of another device), HG_ERR_CUDA
 * (device lookup or launch failed).
 */
int hg_gather_static(int tp, int shard_cols, const void *const *shard_ptrs,
                     void *const *out_ptrs, int M, int *status_out, hg_stream_t stream);

/* Sampler statistics of one gathered row (over its V bf16 values x_c). */
typedef struct hg_row_stats {
  float max_logit;  /* max_c x_c */
  int argmax;       /* smallest c with x_c == max_logit */
  float sum_exp;    /* sum of exp(x_c - max_logit) over x_c != -inf */
  float logsumexp;  /* max_logit + log(sum_exp) */
} hg_row_stats;

/*
 * hg_gather_stats - hg_gather plus sampler statistics of every gathered row,
 * folded where each unit is pushed and reduced per row inside the same kernel. The API page's module docstring
 * notes that the sentinel rewrite leaves every value a sampler uses
 * unchanged, so these are the sampler's statistics of the gathered row. Same
 * arguments, contract and errors as hg_gather (tp <= 16), plus
 *
 *   stats  device pointer to M hg_row_stats, written in stream order: for
 *          row m, over its V = tp * W bf16 values x_c (rank-order columns),
 *          max_logit = max x_c, argmax = the smallest c attaining it,
 *          sum_exp = sum of exp(x_c - max_logit) over x_c != -inf (fp32,
 *          any summation order), logsumexp = max_logit + log(sum_exp).
 *          Rows holding NaN or +inf give unspecified statistics.
 */
int hg_gather_stats(hg_handle *h, const void *const *shard_ptrs, void *const *out_ptrs, int M,
                    hg_row_stats *stats, hg_stream_t stream);

/*
 * Vocabulary operators: the two ends of a model on one vocab-parallel [V, K]
 * matrix. The pages stop at the logits; these have no counterpart there. The
 * matrix is tp shards of [shard_cols, K] (nn.Linear / nn.Embedding layout,
 * rank r holding the rows of tokens r * shard_cols ...), as the weights of
 * hg_gather_fused are; the token-side matrices ([N, K] hidden states,
 * embeddings, their gradients) are single, replicated ones. All sums are fp32.
 *
 *   hg_vocab_embed       out[n] = scale * table[tokens[n]]
 *   hg_vocab_embed_grad  grad_table[v] (+)= scale * sum of grad_out[n] over the
 *                        n with tokens[n] = v
 *   hg_vocab_loss        z[n][v] = logit_scale * sum_k hidden[n][k] * weight[v][k]
 *                        lse[n] = log sum_v exp z[n][v]
 *                        loss[n] = lse[n] - z[n][targets[n]]
 *   hg_vocab_loss_grad   d[n][v] = grad_loss[n] * (exp(z[n][v] - lse[n]) -
 *                        [v = targets[n]]);  grad_hidden = logit_scale * d weight;
 *                        grad_weight (+)= logit_scale * d^T hidden
 *
 * v runs over the real vocabulary, [0, vocab). When vocab < tp * shard_cols the
 * remaining rows of the last shards are padding: whatever they hold (infinities
 * and NaN too) takes no part in the loss or its gradients, and their gradient
 * rows are zero. The logits are never stored: the loss keeps a running
 * maximum and sum, and the gradient recomputes them a piece of the vocabulary
 * at a time, in the matrix's type.
 *
 * Conventions, beside those at the top of this file:
 *  - Every call is asynchronous on `stream`, allocates nothing, does not wait
 *    for the device and may be captured into a CUDA graph. The calls of one
 *    handle share its workspace: issue them on one stream, or order them with
 *    events.
 *  - The device that was current at hg_vocab_create is current at every call, and
 *    the stream and all pointers are its: with another one current a call answers
 *    HG_ERR_ARG before any device work. (hg_vocab_destroy takes any.)
 *  - Results do not depend on timing: the same inputs give the same bits.
 *  - Token and target arrays are device pointers to N signed integers of
 *    id_bytes (4 or 8) bytes each, naturally aligned.
 *  - ld_*: distance in elements between consecutive rows of a token-side
 *    matrix, >= hidden.
 *  - N = 0 is a call with no rows: gradients of the matrix are still written
 *    (as zeros) unless they are accumulated into.
 */
typedef struct hg_vocab hg_vocab;

/* Element types of the matrix and the token-side matrices. */
enum { HG_BF16 = 0, HG_FP16 = 1, HG_FP32 = 2 };

/* Operators a handle serves (hg_vocab_create's `ops`); embedding needs no
 * workspace and is always served. */
enum { HG_VOCAB_EMBED = 1, HG_VOCAB_EMBED_GRAD = 2, HG_VOCAB_LOSS = 4, HG_VOCAB_LOSS_GRAD = 8 };

/*
 * hg_vocab_create - allocate the workspace of the vocabulary operators
 *
 *   tp           shards, 1 <= tp <= HG_MAX_TP
 *   shard_cols   W, matrix rows per shard, >= 1 (no evenness rule)
 *   vocab        real vocabulary, 1 <= vocab <= tp * shard_cols; 0: tp * shard_cols
 *   hidden       K, >= 1; a multiple of 8 for the loss and its gradient
 *   max_rows     largest N of any later call, >= 1
 *   dtype        HG_BF16, HG_FP16, or HG_FP32 (embedding and its gradient only)
 *   ops          HG_VOCAB_* bits of the operators that will be called
 *   piece_bytes  HG_VOCAB_LOSS_GRAD: bound on the logits' gradient kept at a
 *                time (at least one piece of 256 columns per shard); 0: 512 MB.
 *                The columns of a piece follow from it and max_rows, and are those
 *                of every call: few rows on a handle made for many go piece by piece
 *   out          receives the handle
 *
 * Errors: HG_ERR_ARG (bad sizes or type, size overflow), HG_ERR_CUDA (no
 * device, allocation failure). The handle belongs to the current device.
 */
int hg_vocab_create(int tp, int shard_cols, int vocab, int hidden, int max_rows, int dtype,
                    int ops, size_t piece_bytes, hg_vocab **out);

/* Free the handle; waits for its device first, whichever is current. NULL is a no-op. */
int hg_vocab_destroy(hg_vocab *h);

/* Bytes of device memory the handle holds (0 for NULL). */
size_t hg_vocab_workspace_bytes(const hg_vocab *h);

/* Wait for `stream`, then report the device status: HG_OK, HG_ERR_TIMEOUT (a
 * kernel's bounded wait gave up; results of that call are undefined, and the
 * status is cleared by this call), HG_ERR_ARG (NULL, another device current) or
 * HG_ERR_CUDA. */
int hg_vocab_sync(hg_vocab *h, hg_stream_t stream);

/*
 * hg_vocab_embed - scaled embedding lookup
 *
 *   tokens      N ids; one outside [0, vocab) gives a row of zeros
 *   table_ptrs  tp device pointers to [W, K], rows contiguous
 *   scale       multiplied in fp32, rounded once; 1 copies the rows bit for bit
 *   out         [N, K], row distance ld_out
 *
 * Pointers are aligned to their element; where the table, out and the row
 * distances are 16-byte (or 4-byte) aligned the rows move in such words. Errors,
 * before any device work: HG_ERR_ARG, HG_ERR_ROWS (N above max_rows),
 * HG_ERR_CUDA.
 */
int hg_vocab_embed(hg_vocab *h, const void *tokens, int id_bytes, int N,
                   const void *const *table_ptrs, float scale, void *out, size_t ld_out,
                   hg_stream_t stream);

/*
 * hg_vocab_embed_grad - gradient of the lookup to the table
 *
 *   tokens          N ids as in the lookup; one outside [0, vocab) has no gradient
 *   grad_out        [N, K], row distance ld_grad_out
 *   grad_table_ptrs tp device pointers to [W, K], written
 *   accumulate      0: every row is written, zeros where no token points; 1: the
 *                   sum is added to what a row holds (rounded once), and rows
 *                   without tokens are not touched
 *
 * The tokens are sorted and each row's gradients summed in fp32 in the order of
 * their positions, in runs of fixed length. Errors as hg_vocab_embed.
 */
int hg_vocab_embed_grad(hg_vocab *h, const void *tokens, int id_bytes, int N,
                        const void *grad_out, size_t ld_grad_out, void *const *grad_table_ptrs,
                        float scale, int accumulate, hg_stream_t stream);

/*
 * hg_vocab_loss - LM head and softmax cross entropy without the logits
 *
 *   hidden       [N, K], 16-byte aligned, row distance ld_hidden (a multiple of 8)
 *   weight_ptrs  tp device pointers to [W, K], 16-byte aligned
 *   targets      N ids. A negative one masks its row: loss and lse are 0 and the
 *                row's hidden state has no effect. One >= vocab gives a NaN loss.
 *   loss, lse    N floats each
 *
 * Products are exact in fp32 and accumulated in fp32, 1024 of K at a time on the
 * tensor cores, whose sums lose low bits, the rest in fp32 additions. Errors,
 * before any device work: HG_ERR_ARG (also: the handle was not created for it),
 * HG_ERR_ROWS (N above max_rows), HG_ERR_CUDA.
 */
int hg_vocab_loss(hg_vocab *h, const void *hidden, size_t ld_hidden,
                  const void *const *weight_ptrs, const void *targets, int id_bytes, int N,
                  float logit_scale, float *loss, float *lse, hg_stream_t stream);

/*
 * hg_vocab_loss_grad - gradient of hg_vocab_loss
 *
 *   hidden, weight_ptrs, targets, logit_scale   as given to hg_vocab_loss
 *   lse              N floats, hg_vocab_loss's
 *   grad_loss        N floats, the upstream gradient of each row's loss
 *   grad_hidden      NULL, or [N, K], row distance ld_grad_hidden (a multiple of 8),
 *                    16-byte aligned; zeros in masked rows
 *   grad_weight_ptrs NULL, or tp device pointers to [W, K], 16-byte aligned
 *   accumulate       0: grad_weight is overwritten; 1: the gradient, rounded to the
 *                    matrix's type, is added to what grad_weight holds, piece by
 *                    piece of the vocabulary (each element once)
 *
 * At least one of the two gradients is wanted. A row whose target is negative or
 * >= vocab has no gradient, and its hidden state no effect. The logits are the loss's
 * own. d is rounded to the matrix's type before the two products (its error is that of
 * one rounding per term; up to 64 rows it is kept as two rounded terms, and has none to
 * speak of); both products are summed as the loss's, 1024 terms at a time on the
 * tensor cores and these in fp32 additions, and rounded once. Errors as
 * hg_vocab_loss.
 */
int hg_vocab_loss_grad(hg_vocab *h, const void *hidden, size_t ld_hidden,
                       const void *const *weight_ptrs, const void *targets, int id_bytes,
                       const float *lse, const float *grad_loss, int N, float logit_scale,
                       void *grad_hidden, size_t ld_grad_hidden, void *const *grad_weight_ptrs,
                       int accumulate, hg_stream_t stream);

/*
 * Norm of token-side rows: what stands between a model's last layer and
 * its [V, K] matrix (the hidden states of hg_gather_fused and hg_vocab_loss), and
 * in front of each product before that. The pages start at the logits;
 * this has no counterpart there.
 *
 *   hg_norm_rows       s[n] = x[n] + residual[n], in the handle's type
 *                      rstd[n] = 1 / sqrt(mean_k s[n][k]^2 + eps)
 *                      out[n][k] = s[n][k] * rstd[n] * gain[k]
 *   hg_norm_rows_grad  d[n][k] = gain[k] * grad_out[n][k]
 *                      grad_x[n][k] = rstd[n] * d[n][k] - s[n][k] * rstd[n]^3 *
 *                          mean_j d[n][j] * s[n][j] + grad_sum[n][k]
 *                      grad_gain[k] (+)= sum_n grad_out[n][k] * s[n][k] * rstd[n]
 *
 * grad_x is the gradient of x and of residual alike. All arithmetic is fp32; s is
 * rounded once to the handle's type, and what follows is the norm of the rounded
 * rows, those that the gradient is given. Squares and sums that pass the fp32
 * range (rows of about 1e19) give rows of zeros or NaN; squares below it (1e-19, with an
 * eps as small) lose their bits. Between those the gradient holds for rows of any scale.
 *
 * Conventions as for the vocabulary operators (asynchronous, no allocation, no wait for the
 * device, capturable, the handle's device current at every call and the stream and pointers
 * of that device, the same inputs give the same bits). The gradients of one handle share
 * its workspace: they, and graphs that hold them, run one after another. Calls of hg_norm_rows
 * need none and may overlap. No output overlaps an input or another output, but where that
 * is allowed below: other overlaps are refused (HG_ERR_ARG), but for scales over the gain, which
 * is not looked for. Columns of one wider matrix do not overlap. Where all pointers and row distances are 16-byte (or 4-byte) aligned,
 * rows move in such words.
 */
typedef struct hg_norm hg_norm;

/* A further element type, for hg_norm_rows's out: 8 bits, 4 of exponent. */
enum { HG_E4M3 = 3 };

/*
 * hg_norm_create - the norm of rows of one width
 *
 *   hidden    K, >= 1
 *   max_rows  largest N of any later call, >= 1
 *   dtype     HG_BF16, HG_FP16 or HG_FP32: x, residual, s, gain and the gradients
 *
 * Errors: HG_ERR_ARG, HG_ERR_CUDA. The handle belongs to the current device.
 */
int hg_norm_create(int hidden, int max_rows, int dtype, hg_norm **out);

/* Free the handle; waits for its device first, whichever is current. NULL is a no-op. */
int hg_norm_destroy(hg_norm *h);

/* Bytes of device memory the handle holds (0 for NULL). */
size_t hg_norm_workspace_bytes(const hg_norm *h);

/*
 * hg_norm_rows - sum with the residual, norm, and the output's rounding
 *
 *   x         [N, K], row distance ld_x
 *   residual  NULL (s = x), or [N, K], row distance ld_residual
 *   sum       NULL, or [N, K], row distance ld_sum: receives s. May be x or residual
 *   gain      [K]
 *   eps       >= 0
 *   out       [N, K] of out_type, row distance ld_out; may be x or residual (not
 *             both they and sum, and not in 8 bits), same row distance
 *   out_type  the handle's type, or HG_E4M3
 *   scales    HG_E4M3: [N, blocks] floats, rows contiguous; the values are out * scale
 *   scale_block  HG_E4M3: 0: one scale per row; 128: one per 128 columns (blocks =
 *             ceil(K / 128)). A scale is the largest magnitude of its values over
 *             448, at least 2^-126, and 1 where they are all zero. A value within 2^-20 of
 *             the middle between two 8-bit ones goes to either
 *   rstd      NULL, or N floats
 *
 * Errors, before any device work: HG_ERR_ARG, HG_ERR_ROWS (N above max_rows),
 * HG_ERR_CUDA.
 */
int hg_norm_rows(hg_norm *h, const void *x, size_t ld_x, const void *residual,
                 size_t ld_residual, void *sum, size_t ld_sum, const void *gain, float eps, int N,
                 void *out, size_t ld_out, int out_type, float *scales, int scale_block,
                 float *rstd, hg_stream_t stream);

/*
 * hg_norm_rows_grad - gradient of hg_norm_rows (of its unquantised output)
 *
 *   s, rstd    as hg_norm_rows left them (s: its sum, or x where there was no residual)
 *   grad_out   [N, K], row distance ld_grad_out
 *   grad_sum   NULL, or [N, K], row distance ld_grad_sum: gradient that reaches s by
 *              the residual stream
 *   grad_x     NULL, or [N, K], row distance ld_grad_x; may be grad_out or grad_sum,
 *              same row distance
 *   grad_gain  NULL, or [K]
 *   accumulate 0: grad_gain is overwritten; 1: the sum is added to what it holds
 *              (rounded once)
 *
 * At least one of grad_x and grad_gain is wanted. The order of the sum over rows
 * follows from the sizes and alignments alone. N = 0 writes zeros to grad_gain unless it
 * is added to. Errors as hg_norm_rows.
 */
int hg_norm_rows_grad(hg_norm *h, const void *s, size_t ld_s, const void *gain, const float *rstd,
                      const void *grad_out, size_t ld_grad_out, const void *grad_sum,
                      size_t ld_grad_sum, int N, void *grad_x, size_t ld_grad_x, void *grad_gain,
                      int accumulate, hg_stream_t stream);

/*
 * Beam search: what follows the gather where several continuations of a sequence
 * are kept. The pages leave the logits to the caller; this has no counterpart there.
 *
 *   hg_beam_select   total = score[beam] + logit - logsumexp of the beam's logits;
 *                    the `picks` largest over the beams and vocabulary of an item
 *   hg_beam_reorder  state row j of an item takes what row parents[j] holds
 *
 * An item is one sequence of `beams` beams; its rows of the logits, scores and states
 * are neighbours (row = item * beams + beam).
 *
 * Totals are sums in 64 bits of an fp32 score, the logit and a logsumexp that is given in fp32
 * or computed (see lse), and are compared so. Equal totals: the lower beam first; within a beam
 * the larger logit, then the lower token. A total that is NaN, or rounds to -inf in
 * fp32, is no candidate, so a score of -inf takes its beam out of the search (as all
 * but one beam of an item at the first step, whose rows are the same).
 *
 * Conventions as for the vocabulary operators (asynchronous, no allocation, no
 * wait, capturable, one device, same bits). Calls of hg_beam_select of one handle share
 * its workspace: they, and graphs that hold them, run one after another. hg_beam_reorder
 * needs none: its calls may overlap, on other states.
 */
typedef struct hg_beam hg_beam;

#define HG_MAX_BEAMS 64  /* beams of an item */
#define HG_MAX_PICKS 128 /* picks of an item */

/*
 * hg_beam_create - the workspace of a beam search
 *
 *   max_items  largest number of items of any later call, >= 1
 *   beams      1 to HG_MAX_BEAMS
 *   vocab      V, >= 1
 *   picks      1 to HG_MAX_PICKS, at most beams * vocab
 *   dtype      HG_BF16, HG_FP16 or HG_FP32: the logits
 *
 * Errors: HG_ERR_ARG, HG_ERR_CUDA. The handle belongs to the current device.
 */
int hg_beam_create(int max_items, int beams, int vocab, int picks, int dtype, hg_beam **out);

/* Free the handle; waits for its device first, whichever is current. NULL is a no-op. */
int hg_beam_destroy(hg_beam *h);

/* Bytes of device memory the handle holds (0 for NULL). */
size_t hg_beam_workspace_bytes(const hg_beam *h);

/*
 * hg_beam_select - the best continuations of each item
 *
 *   logits    [items * beams, vocab], row distance ld_logits >= vocab (a rank's output
 *             of hg_gather); -inf rules a token out
 *   lse       NULL: computed here, of the logits that are not -inf (a row that holds
 *             NaN or +inf then has no candidates), as a sum of fp32 exponentials in an order
 *             that depends on where the row lies and on the other rows: off by at most 2^-17 +
 *             vocab * 2^-32 (5e-7 measured), so that beams whose totals are closer than that,
 *             or alike, come in any order; or one float per row, lse_stride
 *             floats apart (logsumexp of hg_row_stats: &stats->logsumexp, 4)
 *   scores    items * beams floats
 *   finished  NULL, or items * beams bytes: a beam whose byte is not 0 has one
 *             candidate, the token `end` with the beam's score as it is (its logits
 *             are not read)
 *   end       a token in [0, vocab), or -1 (none; finished is NULL then)
 *   tokens, parents  [items, picks] signed integers of id_bytes (4 or 8) bytes, best first
 *   picked    [items, picks] floats: the totals
 *   picked_finished  NULL, or [items, picks] bytes: 1 where the token is `end` or the
 *             parent was finished, else 0
 *
 * With picks = beams, picked, picked_finished and parents are the next step's
 * scores, finished and reordering (tokens, hg_vocab_embed's input); with picks = 2 * beams
 * there are beams of them that do not end. Where fewer candidates are left, the last
 * picks have token and parent -1, total -inf and are not finished. No output overlaps an
 * input or another output: refused, but for outputs over lse, which are not looked for. An item with more than 1000 candidates at the last
 * pick that cannot be told apart in fp32 takes a path that reads its rows again for every bit of the
 * order, milliseconds instead of microseconds: equal logits (a row of zeros), or a beam whose
 * score is far beyond the others' (-1e9; -inf takes a beam out at no cost).
 *
 * Errors, before any device work: HG_ERR_ARG, HG_ERR_ROWS (items above max_items),
 * HG_ERR_CUDA.
 */
int hg_beam_select(hg_beam *h, const void *logits, size_t ld_logits, const float *lse,
                   size_t lse_stride, const float *scores, const uint8_t *finished, int end,
                   int items, void *tokens, void *parents, int id_bytes, float *picked,
                   uint8_t *picked_finished, hg_stream_t stream);

/* One state of the beams: for every row `outer` x `pieces` runs of piece_bytes bytes,
 * run (o, p) of row r at data + o * outer_stride + r * row_stride + p * piece_stride
 * (all in bytes). A cache [layers, rows, heads, length, width] of which t positions are
 * filled: outer = layers, pieces = heads, piece_bytes = t * width * element. */
typedef struct hg_beam_state {
  void *data;
  size_t outer, outer_stride, row_stride, pieces, piece_stride, piece_bytes;
} hg_beam_state;

#define HG_MAX_STATES 256 /* states of one call */

/*
 * hg_beam_reorder - states follow their beams, in place
 *
 *   parents   items * beams signed integers of id_bytes (4 or 8) bytes: parents[item *
 *             beams + j] is a beam of the same item. One outside [0, beams)
 *             leaves its row as it is. They lie outside the states (else refused)
 *   states    n_states records; the rows of a state and the states do not overlap (a state
 *             listed twice is refused; states that share a part of their runs are not
 *             looked for)
 *
 * All rows of an item take their parents' contents as they were before the call. Only
 * rows that change are written. Errors, before any device work: HG_ERR_ARG (also:
 * runs of one state that overlap by their strides), HG_ERR_ROWS, HG_ERR_CUDA.
 */
int hg_beam_reorder(hg_beam *h, const void *parents, int id_bytes, int items,
                    const hg_beam_state *states, int n_states, hg_stream_t stream);

/* Human-readable text of a status code; never NULL. No counterpart on the
 * pages (HeadGather reports failures as Python exceptions). */
const char *hg_strerror(int status);

#ifdef __cplusplus
}
#endif

#endif /* HG_H_ */
