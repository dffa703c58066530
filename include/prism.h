/*
 * prism.h -- C ABI of the B200 (sm_100a) implementation of Prism's
 * spectral-aware block-importance estimator and the causal block-sparse
 * attention prefill that consumes its mask.
 *
 * Method: "Prism: Spectral-Aware Block-Sparse Attention" (Wang et al., 2026,
 * arXiv 2602.08426).  Passages cited below:
 *   [review:method]  paper.rainbus.top review, the paragraph listing the full
 *                    pipeline, steps (1)-(7);
 *   [review:repro]   the same page, reproducibility paragraph (B = 128,
 *                    d_high = 64, d_low = 96, p = 0.95 / 0.93);
 *   [summary:1], [summary:2A], [summary:2B]  gist.science Technical Summary,
 *                    sections 1 (mean pooling as coarse proxy, block-sparse
 *                    attention computes a subset of blocks), 2A (dual band),
 *                    2B (RMS-based temperature calibration).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - All tensor arguments are DEVICE pointers owned by the caller, contiguous,
 *   16-byte aligned (the mask: 4-byte aligned, so the rows of any group of
 *   heads can be addressed inside a larger mask).  The library never
 *   allocates device memory, never synchronises, and enqueues all work on
 *   the caller's `stream` (0 = the legacy default stream).  Calls are asynchronous: a 0 return means the work
 *   was enqueued, not that it finished.
 * - Layouts (b = batch, hq / hkv = query / key-value heads, N = seqlen (the
 *   padded length when per-sequence lengths are given), D = head_dim = 128,
 *   nb = ceil(N / 128), W = ceil(nb / 32)):
 *     q, o        bf16 [b, hq,  N, D]     (Q after RoPE; output O)
 *     k, v        bf16 [b, hkv, N, D]     (K after RoPE)
 *     mask        uint32 [b, hq, nb, W]:  bit (j % 32) of word j / 32 of row i
 *                 set <=> key block j is kept for query block i.  The
 *                 estimator writes every word (bits j > i are 0).
 * - GQA: query head h reads key/value head h / (hq / hkv).
 * - Return value: PRISM_OK (0) or a negative PRISM_ERR_* code.  Argument
 *   checks run on the host before anything is enqueued; on an error nothing
 *   is enqueued and no output is touched.  The library never aborts or traps.
 */
#ifndef PRISM_B200_H
#define PRISM_B200_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* prism_stream_t; /* == cudaStream_t */

enum {
  PRISM_OK = 0,
  PRISM_ERR_NULL = -1,        /* a required pointer is NULL                        */
  PRISM_ERR_SHAPE = -2,       /* batch/heads/seqlen non-positive, hq % hkv != 0,
                                 or sizes overflow                                 */
  PRISM_ERR_ALIGN = -3,       /* a tensor pointer is not 16-byte aligned (mask: 4)  */
  PRISM_ERR_BAND = -4,        /* band index out of [0, head_dim), duplicated, or an
                                 empty band                                        */
  PRISM_ERR_P = -5,           /* p is not in (0, 1] (p > 1 is treated as 1), or NaN */
  PRISM_ERR_UNSUPPORTED = -6, /* head_dim != 128, block != 128, causal != 1, or an
                                 unknown tau_mode                                  */
  PRISM_ERR_WORKSPACE = -7,   /* workspace NULL or smaller than prism_workspace_size */
  PRISM_ERR_CUDA = -8,        /* a CUDA runtime call failed (launch, attribute)     */
  PRISM_ERR_DEVICE = -9,      /* the device is not sm_100 (B200-class)              */
  PRISM_ERR_TIMEOUT = -10,    /* a kernel gave up a bounded wait (device error word) */
  PRISM_ERR_TAU = -11,        /* PRISM_TAU_EXPLICIT with a temperature that is not
                                 finite and > 0                                    */
  PRISM_ERR_SCRATCH_LIMIT = -12, /* prism_estimate_noalloc: the problem needs more
                                 scratch than prism_noalloc_scratch_bytes()        */
  PRISM_ERR_CACHE = -13       /* a kernel met a length, slot or page number outside
                                 the cache, or a step that does not fit in it
                                 (device error word; state_out of the plan)        */
};

enum {
  PRISM_TAU_RMS = 0,      /* tau_z from the pooled RMS energies (reading R1 below) */
  PRISM_TAU_EXPLICIT = 1  /* tau_hi / tau_lo taken from the config (tests, ablations) */
};

/*
 * Problem statement of one attention layer ([review:method]; [review:repro]).
 * Band sets are HOST arrays of distinct dimension indices in [0, head_dim);
 * the default Prism split for the half-split RoPE layout is
 *   band_hi = {0..31} u {64..95}   (d_high = 64: the 32 fastest RoPE pairs)
 *   band_lo = {16..63} u {80..127} (d_low  = 96: the 48 slowest RoPE pairs)
 * The library copies what it needs during the call; the arrays may be freed
 * when the call returns.
 *
 * tau (step 4 of [review:method]) -- reading R1:
 *   tau_z = RMS(Qbar_z) * RMS(Kbar_z) / (RMS(Qbar_full) * RMS(Kbar_full)),
 *   per (batch, query head), RMS over all pooled blocks and the band's dims,
 *   Kbar of the head's KV head; tau_z = 1 if any RMS is 0.
 * Scores (step 5): L_z[i][j] = Qbar_z[i] . Kbar_z[j] / (tau_z sqrt(d_z)), j <= i.
 * Top-P (step 6): per row and band, keys ranked by (-prob, j); block j kept iff
 *   the mass ranked strictly ahead of it is < p (the crossing block is kept);
 *   p >= 1 keeps every causal block.  Union (step 7): M = M_hi | M_lo.
 */
typedef struct prism_config {
  int batch;
  int hq;
  int hkv;
  int seqlen;
  int head_dim;          /* must be 128 */
  int block;             /* B; must be 128.  seqlen need not be a multiple of B:
                            nb = ceil(seqlen / B) blocks, the last one short; its
                            pooled value is the mean over the tokens it has, and
                            attention sees only real tokens (causal) */
  const int32_t* band_hi;
  int n_hi;
  const int32_t* band_lo;
  int n_lo;
  float p;               /* Top-P threshold, 0 < p; p >= 1 keeps all causal blocks */
  int causal;            /* must be 1 */
  int tau_mode;          /* PRISM_TAU_RMS or PRISM_TAU_EXPLICIT */
  float tau_hi;          /* used only with PRISM_TAU_EXPLICIT; must be > 0 */
  float tau_lo;
  float softmax_scale;   /* attention scale; <= 0 selects 1/sqrt(head_dim) */
  int force_blocks;      /* 0: the mask is exactly M_high | M_low (the method).
                            Optional additions, OR-ed bit flags:
                            PRISM_FORCE_SINK keeps key block 0 in every row,
                            PRISM_FORCE_DIAG keeps the diagonal block j = i.
                            Other bits: PRISM_ERR_UNSUPPORTED. */
  const int32_t* seqlens;  /* NULL: every batch element holds seqlen tokens.
                            Else a host array of batch lengths, 1 <= seqlens[b]
                            <= seqlen (batch <= 256, else
                            PRISM_ERR_UNSUPPORTED; out of range:
                            PRISM_ERR_SHAPE): batch element b holds seqlens[b]
                            tokens at positions 0 .. seqlens[b]-1 of the
                            [.., seqlen, 128] layout, the rest is padding that
                            must hold zeros in q and k and finite values in v.
                            Each sequence has its own ceil(seqlens[b] / B)
                            blocks, pooling, temperatures and Top-P rows; mask
                            rows past them are written as zeros, o rows past
                            them are not written.  Read during the call only. */
} prism_config;

enum { PRISM_FORCE_SINK = 1, PRISM_FORCE_DIAG = 2 };

/*
 * Device workspace, in bytes, that prism_estimate / prism_prefill need for
 * `cfg` (prism_sparse_attn needs none).  Host-only; enqueues nothing.
 * Writes the size to *bytes.  The workspace holds the pooled Q/K means (three
 * bf16 terms per value),
 * per-block energy partials, the temperatures, the fp32 band scores
 * (b * hq * 2 * nb(nb+1)/2 floats) and the estimator's work-queue counters,
 * which each call clears with a memset on its stream; its contents on return
 * are unspecified.
 */
int prism_workspace_size(const prism_config* cfg, size_t* bytes);

/*
 * Optional copies of the estimator's intermediate values, for checking each
 * step on its own (the paper has no counterpart: these are test outputs).
 * Every member may be NULL (not written); all are DEVICE pointers, fp32,
 * owned by the caller, 16-byte aligned (tau: 4-byte).  nb(nb+1)/2 = T.
 *   scores   [b, hq, 2 (hi, lo), T]: the scaled band logits of step (5),
 *            L_z[i][j] = Qbar_z[i] . Kbar_z[j] / (tau_z sqrt(d_z)), in packed
 *            lower-triangular rows (row i starts at i(i+1)/2, j = 0..i).
 *   weights  [b, hq, 2, T], same packing: the unnormalised softmax weights
 *            e_j = 2^((L_j - max_k L_k) log2 e) in (0, 1] exactly as the Top-P
 *            step ranks and sums them (step (6): block j is kept iff the sum
 *            of round(e_k 2^31) over the blocks ranked ahead of it, by (-e, k),
 *            is below max(floor(p Z), 1), Z the row's sum of round(e_k 2^31)).
 *            Written only when p < 1.
 *   tau      [b, hq, 2] = (tau_hi, tau_lo) of step (4).
 *   pooled   [b hq + b hkv, nb, 128]: the block means of step (2) over all
 *            128 dims (rows: the b hq query heads batch-major, then the b hkv
 *            key heads batch-major); a short last block is the mean over its
 *            tokens; blocks past a sequence (per-sequence lengths) are not
 *            written.
 */
typedef struct prism_debug {
  float* scores;
  float* weights;
  float* tau;
  float* pooled;
} prism_debug;

/*
 * Estimator, steps (1)-(7) of [review:method]: band slicing and mean pooling
 * per block of B = 128 tokens, RMS energy of each pooled band, temperatures,
 * dual-band pooled softmax scores, Top-P per query-block row and band, union.
 *   q, k        inputs (layouts above)
 *   mask        output, uint32 [b, hq, nb, W]; every word written
 *   workspace   >= prism_workspace_size(cfg) bytes, 256-byte aligned
 *   dbg         optional (NULL: none) debug outputs, see prism_debug; the
 *               struct is read during the call only
 */
int prism_estimate(const prism_config* cfg, const void* q, const void* k, uint32_t* mask,
                   void* workspace, size_t workspace_bytes, prism_stream_t stream,
                   const prism_debug* dbg);

/*
 * Causal block-sparse attention ([summary:1]: only the selected blocks are
 * computed).  For a query token t in block i it attends to all keys of the
 * kept blocks j < i and to keys s <= t of block i if block i is kept;
 * O_t = sum_s softmax_s(q_t . k_s * scale) v_s, fp32 accumulation, bf16 out.
 * Bits of j > i are ignored; a query block with no kept block gets O = 0.
 * Runs on the tensor cores (tcgen05 MMA, accumulators in tensor memory).
 */
int prism_sparse_attn(const prism_config* cfg, const void* q, const void* k, const void* v,
                      const uint32_t* mask, void* o, prism_stream_t stream);

/*
 * One prefill layer: prism_estimate followed by prism_sparse_attn on the same
 * stream, no host synchronisation in between.  mask_out may be NULL, in which
 * case the mask lives in the workspace (the size then includes it).  The
 * attention is launched with programmatic serialization: its thread blocks
 * may start on SMs the estimator has left, each waiting (bounded, then
 * PRISM_ERR_TIMEOUT through prism_get_last_device_error) until the estimator
 * has published the mask rows it reads, so attention on finished rows
 * overlaps the end of the estimator (Prism: Spectral-Aware Block-Sparse
 * Attention, gist.science Technical Summary, introduction: the cost of
 * finding the relevant blocks is what such methods must keep small).  The
 * outputs equal those of the two separate calls.
 */
int prism_prefill(const prism_config* cfg, const void* q, const void* k, const void* v,
                  uint32_t* mask_out, void* o, void* workspace, size_t workspace_bytes,
                  prism_stream_t stream);

/*
 * Allocation-free estimator.  The paper has no counterpart to this entry
 * point: it exists for callers that cannot allocate device memory -- for
 * example a plugin inside a host framework that hands out no workspace, or a
 * serving loop that forbids cudaMalloc after start-up because it can
 * synchronise the device and fail under memory pressure.
 *
 * Computes exactly what prism_estimate computes (same kernels, same mask,
 * bit for bit) but uses scratch built into the library: a fixed device array
 * of prism_noalloc_scratch_bytes() = 32 MiB that every GPU loading the library
 * holds until the process exits.  The caller still passes q, k and mask
 * (device pointers, layouts as above); no dbg outputs.
 *   - Problems whose estimator workspace (prism_workspace_size less the
 *     mask slot only prism_prefill uses) exceeds 32 MiB are rejected with
 *     PRISM_ERR_SCRATCH_LIMIT before anything is enqueued (the Llama-3-8B
 *     shape, 32 Q / 8 KV heads, batch 1, fits up to 265 blocks = 33,920
 *     tokens).
 *   - The first call on a device looks up the array's device address with
 *     cudaGetSymbolAddress while that device is current; make that first call
 *     before any stream capture.
 *   - Calls no cudaMalloc, cudaFree or other allocating routine.
 *   - Every call on a device shares the one array, which keeps the previous
 *     call's contents; the few counters that must start at zero are cleared
 *     on `stream` at the start of each call.  Calls whose work overlaps on
 *     the GPU (different streams, or host threads, without ordering between
 *     them) race on the array.  Order them on one stream, or synchronise
 *     between them.
 */
int prism_estimate_noalloc(const prism_config* cfg, const void* q, const void* k, uint32_t* mask,
                           prism_stream_t stream);

/* Size in bytes of the scratch built into prism_estimate_noalloc. */
size_t prism_noalloc_scratch_bytes(void);

/*
 * Paged 8-bit key/value cache
 * ---------------------------
 * What follows a prefill: K and V of every request stay in pages of e4m3
 * codes, and new tokens -- one a request while it decodes, a few when drafted
 * tokens are verified, thousands when a prompt goes on -- attend over them.
 * A step is three calls on one stream, with no host synchronisation between
 * them and nothing read back, so it can be captured into a graph and replayed:
 *
 *   prism_cache_plan    request lengths -> pages, packed row offsets, slots
 *   prism_cache_store   K and V rows of the new tokens -> codes and scales
 *   prism_cache_attn    Q rows of the new tokens -> O over the requests' pages
 *
 * Layouts (n = requests, P = page, T = tokens, a packed buffer's rows):
 *   k_cache, v_cache  e4m3 codes, page p at p * page_stride bytes,
 *                     [hkv, P, 128] inside a page
 *   k_scale, v_scale  fp32 [num_pages, hkv]: a code c of page p and head h
 *                     stands for c * scale[p, h].  Scales are powers of two
 *                     >= 2^-64; a request's V scales lie within 2^80 of each
 *                     other (weights are taken times their page's scale in 32
 *                     bits; an all-zero page, 2^-64, beside values up to 2^24)
 *   table             int32 [n, max_pages]: the pages of each request in the
 *                     order of its tokens; entries behind a request's last
 *                     page are not read
 *   lens              int32 [n]: tokens of each request, the new ones included
 *   starts            int32 [n + 1]: the new tokens of request i are the rows
 *                     starts[i] .. starts[i + 1] - 1 of the packed buffers
 *   slots             int32 [T]: page * P + place in the page of each packed
 *                     row, -1 for a row that no request has
 * Lengths live on the device, so only the kernels can check them: what lies
 * outside the cache is left out (below) and reported as PRISM_ERR_CACHE
 * through prism_get_last_device_error.
 */
typedef struct prism_cache_config {
  int requests;        /* n, 1 .. 4096 */
  int page;            /* tokens per page: 16, 32, 64 or 128 */
  int num_pages;       /* pages of the cache; num_pages * page < 2^31 */
  int max_pages;       /* row length of table; max_pages * page < 2^31 */
  int hq;              /* hq % hkv == 0, hq / hkv <= 64 */
  int hkv;
  int head_dim;        /* must be 128 */
  int tokens;          /* T: rows of the packed buffers (a capacity: rows behind
                          starts[n] are padding) */
  int max_add;         /* most new tokens a request is expected to bring, 1 .. T.
                          Chooses between kernels and working sizes: plans and
                          stores do not depend on it, attention only in its
                          rounding; more tokens than expected are slower, not
                          wrong */
  float softmax_scale; /* attention scale; <= 0 selects 1/sqrt(head_dim) */
  long long page_stride; /* bytes between pages in k_cache and v_cache, a multiple
                          of 16 and >= hkv * page * 128; 0 selects that size
                          (pages side by side) */
} prism_cache_config;

/*
 * Plan of a step.  All pointers are device pointers (int32, 4-byte aligned).
 *   held  [n]  tokens that each request has
 *   add   [n]  tokens that it brings now; 0: none; -1: the request is over and
 *              its pages are returned
 *   ring  [num_pages]  ring of free pages: `count` of them from place `head` on
 *   state [4]  {head, count, 0, -}
 * A request's tokens fill its begun page first; opened pages are taken from the
 * ring's head in request order and entered into table, returned ones go
 * behind its last free page and can be taken from the next call on.  Writes
 *   table      entries of the opened pages (a returned request's row keeps its
 *              entries, which nothing reads)
 *   lens, starts, slots   for prism_cache_store and prism_cache_attn
 *   state_out  [4]  {head, count, 0, status}: status 0, or PRISM_ERR_CACHE
 * lens may be held and state_out may be state (a step in place).  Word 2 of
 * state_out must be 0 before the call.
 * A step that does not fit -- more new tokens than T, more pages than the ring
 * has, a request longer than max_pages * page, a length < 0, a begun page that
 * is not one of the cache's -- changes nothing: lens = held, starts all 0,
 * every slot -1, ring, table and state as they were, status PRISM_ERR_CACHE.
 * A ring entry that is no page number gives slots of -1 and the same status.  A
 * returned request's entry that is none goes into the ring as it is and sets the
 * device error word alone.
 */
int prism_cache_plan(const prism_cache_config* cfg, const int32_t* held, const int32_t* add, int32_t* ring,
                     const int32_t* state, int32_t* table, int32_t* lens, int32_t* starts, int32_t* slots,
                     int32_t* state_out, prism_stream_t stream);

/*
 * Stores K and V of T rows (bf16; row t of head h at t * tok + h * head
 * elements, strides multiples of 8, 16-byte aligned; strides of 0 select the
 * packed [T, hkv, 128]) at their slots; rows of slot -1 are skipped.
 *   s = 2^max(-64, ceil(log2(amax / 448))), amax over the finite new values of
 *   a page and head.  A page written from its first place gets scale s.  A
 *   page begun before keeps the larger of its scale and s; if that grows, its
 *   older codes c become e4m3(c * old / new) (exact but for codes that become
 *   subnormal).  New codes are e4m3(x / scale), to nearest even; a NaN or
 *   infinite x is stored as NaN.
 * The slots of one page are consecutive rows in ascending order, as
 * prism_cache_plan makes them.  Places that no row has are left as they were.
 * A slot outside the cache is skipped and reported.
 */
int prism_cache_store(const prism_cache_config* cfg, const void* k, long long k_tok, long long k_head, const void* v,
                      long long v_tok, long long v_head, const int32_t* slots, void* k_cache, void* v_cache,
                      float* k_scale, float* v_scale, prism_stream_t stream);

/*
 * Device workspace, in bytes, of prism_cache_attn for cfg.  Host-only.  Its
 * contents need not be kept or cleared between calls; two calls that may run
 * at the same time need two workspaces.
 */
int prism_cache_workspace_size(const prism_cache_config* cfg, size_t* bytes);

/*
 * Attention over the cache: row starts[i] + t of request i sees the tokens at
 * positions <= lens[i] - (starts[i + 1] - starts[i]) + t of its pages,
 *   O = sum_s softmax_s(q . k_s * scale) v_s,
 * query head h reading KV head h / (hq / hkv); fp32 accumulation and softmax,
 * bf16 q and O.  K and V enter the tensor cores as they are stored; q as two
 * 8-bit terms (its 8 bits, down to 2^-17 of the row's largest), a weight in 11
 * bits (one rounding to fp16, whose smallest step is at most 2^-28 of the row's
 * largest weight times V scale).  Requests of up to 64 rows (new tokens x hq /
 * hkv) and of more go to different kernels of the same call, unless max_add says
 * that there are none of more, or all of those together are little work (the sum
 * over them of ceil(rows / 32) * (ceil(lens / 128) + 9) * hkv is at most 4000):
 * then the kernel for few takes them too.  So the last bits of a request's O may
 * depend on the rest of the call.
 *   q     bf16, row t of head h at t * q_tok + h * q_head elements (multiples
 *         of 8; 0, 0 selects [T, hq, 128])
 *   mask  optional uint32 [n, hq, W], W = ceil(ceil(max_pages * page / 128) /
 *         32): bit (j % 32) of word j / 32 set <=> query head h of request i
 *         attends to the tokens 128 j .. 128 j + 127 (the mask row of
 *         prism_estimate).  NULL: to all.  Blocks that no head of a KV head's
 *         group keeps are not read.
 *   o     bf16 [T, hq, 128]; rows of no request are left as they were
 * A row that sees no token gets O = 0.  A length below 0 or above max_pages *
 * page, and starts that descend or leave 0 .. T, are clamped and reported;
 * more rows than tokens are no error.  Tokens of a table entry that is no page
 * number are left out and reported; entries of blocks that are not read
 * may be anything.  Cache places behind a request's last token are never used,
 * whatever they hold.
 */
int prism_cache_attn(const prism_cache_config* cfg, const void* q, long long q_tok, long long q_head,
                     const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                     const int32_t* table, const int32_t* lens, const int32_t* starts, const uint32_t* mask, void* o,
                     void* workspace, size_t workspace_bytes, prism_stream_t stream);

/*
 * Reads and clears the device error word that kernels set when a bounded
 * wait gives up (PRISM_ERR_TIMEOUT) or cache data is invalid
 * (PRISM_ERR_CACHE) -- synchronises `stream` first.  Returns PRISM_OK when no
 * kernel reported an error, a PRISM_ERR_* code otherwise.
 */
int prism_get_last_device_error(prism_stream_t stream);

/*
 * Diagnostic for the failure path (the paper has no counterpart): enqueues a
 * one-warp kernel on `stream` that waits, with the same bounded-wait helpers
 * the estimator and attention kernels use but a limit of `timeout_us`
 * microseconds (1 .. 2,000,000), on a device word nothing writes and on an
 * mbarrier phase nothing completes.  Both waits give up and record
 * PRISM_ERR_TIMEOUT; the kernel returns normally, so the context stays usable.
 * Read the result with prism_get_last_device_error(stream), which then returns
 * PRISM_ERR_TIMEOUT (and clears it).  Returns PRISM_OK once enqueued,
 * PRISM_ERR_SHAPE for a timeout out of range, PRISM_ERR_DEVICE / _CUDA.
 */
int prism_selftest_wait_timeout(prism_stream_t stream, unsigned timeout_us);

/* Static description of a status code; never NULL. */
const char* prism_status_str(int status);

/* Library version as MAJOR * 10000 + MINOR * 100 + PATCH. */
int prism_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PRISM_B200_H */
