/*
 * gdn.h -- C ABI of libgdn: the chunkwise (64-token) Gated Delta Network
 * prefill core on NVIDIA GB300 (sm_103a), dense and event-sparse forms, and the
 * decode step of softmax-attention layers beside it (paged cache, one-token
 * attention, sampling; "Decode step" below) with their prompt chunks (rotary
 * positions, attention of new tokens, log probabilities; "Prompt chunks" below).
 *
 * Source of the operator: "SparseGDN: Chunk Sparse in Linear Attention"
 * (arXiv 2610.41420v1), as paraphrased by its Chinese reading notes:
 *   Sec. 2.1, Eqs. 1-4   dense chunkwise recurrence and chunk output
 *   Sec. 2.3, Eqs. 5-9   local Delta system, block-adjacent solver, Tail-16 score
 *   Sec. 2.5, Eqs. 15-16 deferred W, CSR event layout, device-resident event count
 *   Sec. 2.6, Eqs. 17-21 event-sparse propagation and prefix-gap recovery
 *   Sec. 2.7, Eqs. 22-25 two-chunk group output from compact state snapshots
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Shapes.  B sequences of T tokens; Nq query/key heads of width d; Nv = 2*Nq
 * value heads of width dv.  Value heads 2p and 2p+1 form head pair p and read
 * query/key head p.  C = ceil(T/64) chunks (a partial last chunk holds the
 * remaining T - 64 (C-1) tokens), G = ceil(C/2) output groups, P = Nq pairs.
 * This version requires d == dv == 128 and C <= 16384 (T == 0 and B == 0 are
 * accepted).
 *
 * Layouts (row-major, contiguous, innermost last):
 *   q, k      [B, T, Nq, d]      dtype (bf16 or fp32)
 *   v, o      [B, T, Nv, dv]     dtype
 *   beta      [B, T, Nv]         fp32, per-token update strength
 *   g         [B, T, Nv]         fp32, log2 retention accumulated inside each
 *                                64-token chunk, inclusive of the token's own
 *                                gate (the pages' g_{c,h,i})
 *   mask      [B, P, C]          uint8 0/1 event mask, shared by a head pair
 *   h0, s_final [B, Nv, d, dv]   fp32 recurrent state (key dim x value dim)
 *   score     [B, Nv, C]         fp32 Tail-16 write score s_{c,h} (Eq. 9)
 *   O is the GDN-core output before RMSNorm, output gate and projection,
 *   scaled by 1/sqrt(d).
 *
 * Memory and streams.  Every pointer is a caller-owned DEVICE pointer on the
 * current CUDA device, 16-byte aligned (the workspace: 256-byte aligned).  The
 * library never allocates device memory, never frees and never synchronises,
 * except in the status queries.  Work is enqueued on `stream` (a cudaStream_t;
 * NULL = legacy default stream) and is complete only when that stream is.  The
 * bf16 prefills fork part of their kernels onto library-owned streams (made
 * once per device, at higher priority) with an event recorded on `stream`,
 * and join them back with events before returning, so `stream` alone orders
 * the work; a stream capture of `stream` takes the forked kernels in.  Make
 * the first prefill on a device outside a capture (it creates those streams).
 * Calls on distinct workspaces are independent (concurrent calls share the
 * library's streams, so their forked kernels run one call after the other);
 * two calls that share a workspace must be stream-ordered.  The event count E
 * never leaves the device.
 *
 * Errors.  Argument problems are detected on the host before anything is
 * enqueued and returned synchronously (GDN_ERR_NULL / SHAPE / DTYPE / ALIGN /
 * WORKSPACE / UNSUPPORTED / DEVICE).  A failed launch returns GDN_ERR_CUDA.
 * Conditions only the GPU can see (event or snapshot capacity exceeded, a
 * wait inside a kernel that ran past its time limit) are latched in a device
 * status word; the kernels never write past a capacity and never wait
 * without a limit, and gdn_workspace_status() / gdn_events_status() report
 * the latch.
 */
#ifndef GDN_H
#define GDN_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define GDN_API __attribute__((visibility("default")))
#else
#define GDN_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    GDN_OK = 0,
    GDN_ERR_NULL = 1,        /* a required pointer is NULL */
    GDN_ERR_SHAPE = 2,       /* unsupported or inconsistent sizes */
    GDN_ERR_DTYPE = 3,       /* unknown dtype or solver enum */
    GDN_ERR_ALIGN = 4,       /* a pointer is not 16-byte (workspace: 256-byte) aligned */
    GDN_ERR_WORKSPACE = 5,   /* workspace smaller than gdn_workspace_bytes() */
    GDN_ERR_UNSUPPORTED = 6, /* valid request this library does not implement */
    GDN_ERR_CUDA = 7,        /* a CUDA runtime call or launch failed */
    GDN_ERR_DEVICE = 8,      /* current device is not a compute-capability 10.3 GPU */
    GDN_ERR_CAPACITY = 9,    /* (device-latched) more events or snapshots than capacity */
    GDN_ERR_TIMEOUT = 10     /* (device-latched) a kernel wait exceeded its 2 s limit and was abandoned */
} gdn_status;

/* GDN_E4M3 (8-bit floating point: 4 exponent bits, 3 fraction bits, largest
 * finite value 448) is a storage type of the paged key-value cache only. */
typedef enum { GDN_BF16 = 0, GDN_F32 = 1, GDN_E4M3 = 2 } gdn_dtype;

/* Intra-chunk solver for M = I + A_Delta (Sec. 2.3).
 * EXACT ("Full64"): C = M^-1.  BLOCK_ADJ: only the four diagonal and three
 * sub-diagonal 16x16 blocks of M^-1 are kept (Eq. 7). */
typedef enum { GDN_SOLVER_EXACT = 0, GDN_SOLVER_BLOCK_ADJ = 1 } gdn_solver;

typedef struct {
    int32_t B, T, Nq, Nv, d, dv;
    gdn_dtype dtype; /* storage type of q, k, v, o (and of internal U / W) */
} gdn_shape;

/* CSR event lists (Sec. 2.5).  One row per (sequence b, head pair p), physical
 * row id i = b*P + p.  Rows are ordered by event count descending, ties by
 * physical id ascending ("long chains first"; a caller mask carries no tiers).
 * Events inside a row ascend in chunk index.  All arrays are caller-owned
 * device memory written by gdn_select_events(). */
typedef struct {
    int32_t *row_pair;  /* [B*P]       physical id of row j */
    int32_t *row_ptr;   /* [B*P+1]     offset of row j's first event; row_ptr[B*P] = E */
    int32_t *ev_chunk;  /* [capacity]  chunk index of event e */
    int32_t *grp_pred;  /* [B*P*G]     indexed by physical id: global index of the last
                                       event of that pair with chunk < 2r, or -1 */
    int32_t *snap_slot; /* [capacity]  dense number (in event order) of the events some
                                       group reads as predecessor, else -1 */
    int32_t *counts;    /* [4]         E, number of snapshots, status bits, reserved */
    int32_t capacity;   /* entries available in ev_chunk and snap_slot */
} gdn_events;

/* What gdn_prefill_ex computes: every chunk an event, a caller mask, or events
 * chosen on the GPU from the Tail-W scores (Sec. 2.4). */
typedef enum { GDN_MODE_DENSE = 0, GDN_MODE_SPARSE = 1, GDN_MODE_ONLINE = 2 } gdn_mode;

/* Execution variants (the pages' ablation axes; Secs. 3.4-3.5).  Zero-initialise:
 * every field's zero value is the default.
 *   tail_window  rows of the Tail-W write-score window, the last W rows of a
 *                chunk's U: 0 (= 16), 8, 16, 32 or 64 (Fig. 10).  Changes only
 *                the scores, and through them an online selection.
 *   w_deferred   0: with a mask known up front, W = C-bar K is built inside the
 *                intra step for the event chunks;  1: the intra step stores the
 *                compact C-bar blocks and a separate tensor-core kernel builds W
 *                for the events after compaction (the order online selection
 *                needs).  The results are identical bit for bit (bf16 storage;
 *                fp32 storage always builds W separately).
 *   scan_runs    bf16 storage only.  0: the event scan walks each CSR row once,
 *                the state held on chip for the whole row (every event applied
 *                once);  1: the row is cut into runs of 16 chunks whose affine
 *                maps are built in parallel, chained, then replayed (three
 *                launches; every event applied three times, on tcgen05 tensor
 *                cores).  Both compute the same recurrence (Eqs. 1-2, 17-21);
 *                their fp32 rounding orders differ, so the results agree to
 *                rounding, not bit for bit.  scan_runs = 1 needs the larger
 *                workspace that gdn_workspace_bytes_ex() reports for it.
 *   scan_full    1: the masked full scan, the pages' reference for the CSR
 *                scan (Table 6): the intra step builds W for every chunk and
 *                the scan visits every chunk, computing both products on each
 *                but keeping them on the mask's events only, with the same
 *                decay arithmetic (the gap factors of Eq. 21).  Identical
 *                results bit for bit; more work.  bf16, given mask or dense
 *                (not online selection, not w_deferred, not scan_runs).
 *   states_expanded  1: the pages' reference for compact states and mapped
 *                output (Table 6): the scan writes the entry state of every
 *                two-chunk output group to a slot of its own (dense group
 *                states, B*P*G slots), and the output reads its group's slot
 *                directly instead of the predecessor's compact snapshot
 *                through the group map.  Identical results bit for bit.  bf16,
 *                one-pass scan.
 *   online_split online selection in two calls, for head pairs sharded over
 *                ranks (tensor parallelism: the selection couples a sequence's
 *                16 pairs, Eq. 14).  Both calls use mode GDN_MODE_ONLINE, the
 *                rank's own pairs (any number) and the same workspace.
 *                1: the intra step only; writes `score` (required) and keeps
 *                U and the C-bar blocks in the workspace.  The caller gathers
 *                every rank's scores and chunk gate tails gamma (g at each
 *                chunk's last token) and selects with
 *                gdn_select_events_gamma().  2: the rest of the pipeline
 *                (compaction, deferred W, scan, output) on the workspace of
 *                call 1, with the rank's rows of that selection in `mask`.
 *                The two calls compute what one online prefill computes, bit
 *                for bit.
 *   reserved     must be zero. */
typedef struct {
    int32_t tail_window;
    int32_t w_deferred;
    int32_t scan_runs;
    int32_t scan_full;
    int32_t states_expanded;
    int32_t online_split;
    int32_t reserved[2];
} gdn_options;

/* Bytes of workspace the prefill entry points need for `shape`: sparse = 0
 * gdn_prefill_dense, 1 gdn_prefill_sparse, 2 gdn_prefill_sparse_online (all
 * with default execution variants).  0 for invalid shapes. */
GDN_API size_t gdn_workspace_bytes(const gdn_shape *shape, gdn_solver solver, int sparse);

/* Bytes of workspace gdn_prefill_ex needs for `mode` and the options `opt`
 * (NULL = defaults; equal to gdn_workspace_bytes for the same mode).  Some
 * variants keep extra buffers: w_deferred the compact C-bar blocks, scan_runs
 * the per-run affine maps.  0 for invalid shapes or options. */
GDN_API size_t gdn_workspace_bytes_ex(const gdn_shape *shape, gdn_solver solver, gdn_mode mode,
                                      const gdn_options *opt);

/* Bytes of one device buffer that holds the arrays of a gdn_events for `shape`
 * with room for `capacity` events: row_pair, row_ptr, ev_chunk, grp_pred,
 * snap_slot and counts, in that order, each at a 256-byte aligned offset.
 * 0 for an invalid shape or a negative capacity.  A capacity of B*P*C always
 * suffices (every chunk of every pair an event); the pages' selector bounds E
 * by 16 k_H per sequence (Sec. 2.5). */
GDN_API size_t gdn_events_bytes(const gdn_shape *shape, int32_t capacity);

/* Points the arrays of *events into `buffer` (device memory of at least
 * gdn_events_bytes(shape, capacity) bytes, 256-byte aligned) in the layout
 * gdn_events_bytes() describes, and sets events->capacity.  Host-only: nothing
 * is enqueued and the buffer is not touched.  Returns GDN_ERR_NULL, _SHAPE or
 * _ALIGN on bad arguments. */
GDN_API gdn_status gdn_events_carve(const gdn_shape *shape, int32_t capacity, void *buffer, gdn_events *events);

/* Event compaction (Sec. 2.5, Eq. 16): turn the [B,P,C] 0/1 mask into CSR
 * event lists, the per-group predecessor event and the snapshot numbering.
 * E = sum of the mask stays on the device (counts[0]).  If E > capacity the
 * status bit 1 is set in counts[2], nothing past capacity is written and
 * gdn_events_status() returns GDN_ERR_CAPACITY.  No workspace needed. */
GDN_API gdn_status gdn_select_events(const gdn_shape *shape, const uint8_t *mask,
                             gdn_events *events, void *stream);

/* Online event selection (Sec. 2.4, Eqs. 10-14) for 16 head pairs (Nv == 32):
 * from the Tail-16 scores score [B,Nv,C] (fp32, Eq. 9), the gates g [B,T,Nv]
 * (gamma = g at each chunk's last token) and an optional output-visibility
 * energy eta [B,Nv] (NULL: G_h = 1), choose per sequence the tier of every pair
 * (Eq. 14) and its chunks (anchors 0 and C-1 plus the best k_tier - 2 chunks by
 * the in-pair rank q, Eqs. 10 and 13); writes mask_out [B,16,C] (0/1) and, if
 * non-NULL, tier_out [B,16] (0 low, 1 mid, 2 high).  Ties: q descending then
 * lower chunk; pair gains descending then lower pair; B(x,k) ties take the
 * smaller k.  Workspace: gdn_select_scored_workspace_bytes(shape), 256-byte
 * aligned.  Other head counts return GDN_ERR_UNSUPPORTED. */
GDN_API gdn_status gdn_select_events_scored(const gdn_shape *shape, const float *score, const float *g,
                                    const float *eta, uint8_t *mask_out, int32_t *tier_out,
                                    void *workspace, size_t workspace_bytes, void *stream);
GDN_API size_t gdn_select_scored_workspace_bytes(const gdn_shape *shape);

/* gdn_select_events_scored with the chunk gate tails given directly: gamma
 * [B,Nv,C] fp32 (gamma[b,h,c] = g at chunk c's last token) instead of g
 * [B,T,Nv].  For a selection over head pairs gathered from several ranks
 * (online_split), where each rank holds only its own heads' gates.  Same
 * results as gdn_select_events_scored on the same values.  shape gives B, C
 * (through T) and Nv == 32; workspace as gdn_select_scored_workspace_bytes. */
GDN_API gdn_status gdn_select_events_gamma(const gdn_shape *shape, const float *score, const float *gamma,
                                           const float *eta, uint8_t *mask_out, int32_t *tier_out,
                                           void *workspace, size_t workspace_bytes, void *stream);

/* Synchronises `stream` and reports the status bits of an events struct. */
GDN_API gdn_status gdn_events_status(const gdn_events *events, void *stream);

/* Dense prefill (Secs. 2.1 and 2.3; Eqs. 1-8): every chunk is a recurrent
 * event.  Writes o and s_final (the state after the last chunk, for decoding).
 * h0 may be NULL (zero initial state); score may be NULL. */
GDN_API gdn_status gdn_prefill_dense(const gdn_shape *shape,
                             const void *q, const void *k, const void *v,
                             const float *beta, const float *g, const float *h0,
                             gdn_solver solver, void *o, float *s_final, float *score,
                             void *workspace, size_t workspace_bytes, void *stream);

/* Event-sparse prefill (Secs. 2.3-2.7; Eqs. 5-25).  Runs the whole pipeline on
 * the GPU: intra-chunk solve and Tail-16 score for every chunk, mask -> CSR
 * compaction, deferred W for selected events only, the event scan (read and
 * write only on selected events, decay always), and the two-chunk group
 * output from compact state snapshots.  Selected chunks write U' in place of
 * U; unselected chunks keep U.  mask: [B,P,C] uint8 0/1.  h0 and score may be
 * NULL. */
GDN_API gdn_status gdn_prefill_sparse(const gdn_shape *shape,
                              const void *q, const void *k, const void *v,
                              const float *beta, const float *g, const float *h0,
                              const uint8_t *mask, gdn_solver solver,
                              void *o, float *s_final, float *score,
                              void *workspace, size_t workspace_bytes, void *stream);

/* Event-sparse prefill with online selection, the pages' full pipeline
 * (Secs. 2.3-2.7): intra step (U, Tail-16 scores, compact C-bar), online
 * selection (as gdn_select_events_scored), compaction, deferred W for the
 * selected events only, event scan, group output.  16 head pairs only.
 * score (may be NULL) receives the Tail-16 scores, mask_out (may be NULL) the
 * selected mask [B,16,C], tier_out (may be NULL) the tiers [B,16]; eta may be
 * NULL.  Workspace: gdn_workspace_bytes(shape, solver, 2). */
GDN_API gdn_status gdn_prefill_sparse_online(const gdn_shape *shape,
                                     const void *q, const void *k, const void *v,
                                     const float *beta, const float *g, const float *h0,
                                     const float *eta, gdn_solver solver,
                                     void *o, float *s_final, float *score, uint8_t *mask_out,
                                     int32_t *tier_out, void *workspace, size_t workspace_bytes,
                                     void *stream);

/* The general prefill: `mode` selects dense (mask ignored), sparse (mask
 * required) or online selection (eta, mask_out and tier_out as in
 * gdn_prefill_sparse_online, 16 head pairs); `opt` (NULL = defaults) selects
 * execution variants.  Arguments otherwise as gdn_prefill_sparse; workspace
 * gdn_workspace_bytes_ex(shape, solver, mode, opt).  Unknown option values return
 * GDN_ERR_UNSUPPORTED before anything is enqueued. */
GDN_API gdn_status gdn_prefill_ex(const gdn_shape *shape, gdn_mode mode,
                          const void *q, const void *k, const void *v,
                          const float *beta, const float *g, const float *h0,
                          const uint8_t *mask, const float *eta, gdn_solver solver,
                          const gdn_options *opt, void *o, float *s_final, float *score,
                          uint8_t *mask_out, int32_t *tier_out, void *workspace,
                          size_t workspace_bytes, void *stream);

/* One autoregressive decode step from a state, e.g. the S_final of a prefill
 * (the pages return S_C for the decoding that follows; Sec. 2.6).  It is
 * Eqs. 1-4 for a chunk of a single token whose log2 retention is a:
 *   U' = beta v - beta 2^a S^T k,   S <- 2^a S + k U'^T,
 *   o  = [2^a S^T q + <q,k> U'] / sqrt(d)   (= S_new^T q / sqrt(d)).
 * shape: B sequences, T == 1, Nq, Nv = 2 Nq, d = dv = 128, dtype of q, k, v, o.
 * q, k [B,Nq,d]; v [B,Nv,dv]; beta [B,Nv] fp32; a [B,Nv] fp32: this token's
 * log2 retention (the increment of g; g of a prefill is its within-chunk
 * running sum); state [B,Nv,d,dv] fp32, updated in place; o [B,Nv,dv] out.
 * Value head h reads query/key head h/2.  All device pointers, 16-byte aligned.
 * Enqueues one kernel on `stream`; no workspace. */
GDN_API gdn_status gdn_decode_step(const gdn_shape *shape, const void *q, const void *k, const void *v,
                                   const float *beta, const float *a, float *state, void *o, void *stream);

/* ---- Decode step of the softmax-attention layers ---------------------------
 * A hybrid decoder interleaves the gated delta layers above with softmax
 * attention layers.  Their keys and values grow with the sequence, so they are
 * kept in pages of `page` tokens that requests take from one pool.  Request b
 * holds its tokens in order in the pages its row of the block table names:
 * token j lies in page table[b][j / page], cell j % page, and its slot is
 * table[b][j / page] * page + j % page.  None of these calls waits for the
 * GPU or allocates; all of them may be captured in a CUDA graph.
 *
 * gdn_kv_cache describes one layer's cache.  Element (page, cell, head, i) of
 * both k and v lies at page * stride_page + cell * stride_token +
 * head * stride_head + i elements, so both storage orders (token-major
 * [pages, page, Hkv, d] and head-major [pages, Hkv, page, d]) are taken as they
 * are.  k, v and every stride are multiples of 16 bytes; d is 64, 128 or 256.
 * k_scale, v_scale [Hkv] (GDN_E4M3 only, else NULL): a stored value x stands
 * for x * scale[head]. */
typedef struct {
    void *k, *v;
    int64_t stride_page, stride_token, stride_head; /* in elements */
    const float *k_scale, *v_scale;
    int64_t pages;      /* pages in the pool */
    int32_t page;       /* tokens per page, >= 1 */
    int32_t Hkv, d;
    gdn_dtype dtype;    /* GDN_BF16, GDN_F32 or GDN_E4M3 */
} gdn_kv_cache;

/* Block tables and slot maps of one step, from the requests' lengths.  Request
 * b has c = cached_lens[b] tokens in the cache (cached_lens NULL: 0) and adds
 * new_lens[b] (negative lengths count as 0).  With old = ceil(c / page) and
 * need = min(ceil((c + new) / page), max_pages):
 *   block_table [B][max_pages]  entries below old are kept, entries old..need-1
 *                take the next ids of free_pages [n_free], requests in order
 *                (-1 once the list is used up), entries from need on become -1;
 *   seq_lens [B] c + new;  cu_new [B+1] running sum of the new tokens;
 *   slots [n_slots] (int64) the slot of every new token, requests in order, -1
 *                where it has no page and behind the last token;
 *   positions [n_slots] the token's position in its sequence, 0 behind the last;
 *   counts [4] {new tokens, pages taken, status bits, longest sequence}.
 * Status bits: 1 the free list was too short, 2 a sequence needs more than
 * max_pages pages, 4 more new tokens than n_slots.  Calling again with the same
 * lengths and free list writes the same values.  No output may overlap an input
 * (GDN_ERR_UNSUPPORTED): seq_lens becomes the next step's cached_lens, but not in
 * place. */
GDN_API gdn_status gdn_page_tables(int32_t B, int32_t page, int32_t max_pages, const int32_t *cached_lens,
                                   const int32_t *new_lens, const int32_t *free_pages, int32_t n_free,
                                   int32_t *block_table, int32_t *seq_lens, int32_t *cu_new, int64_t *slots,
                                   int32_t *positions, int32_t n_slots, int32_t *counts, void *stream);

/* Synchronises `stream` and reports the status bits of counts
 * (GDN_ERR_CAPACITY if any is set). */
GDN_API gdn_status gdn_page_tables_status(const int32_t *counts, void *stream);

/* Writes the keys and values of n new tokens into the cache: row t of k and v
 * ([Hkv][d] at t * k_stride_token + head * k_stride_head elements, multiples of
 * 16 bytes; v alike) goes to slot slots[t]; slots outside [0, pages * page) are
 * skipped.  Rows of dtype (GDN_BF16 or GDN_F32) are copied into a cache of the
 * same dtype, or stored in a GDN_E4M3 cache as x / scale[head], rounded to
 * nearest even and saturated at +-448 (NaN stays NaN).  What a slot holds
 * after two rows were written to it is undefined: each 16 bytes are those of
 * either row. */
GDN_API gdn_status gdn_kv_append(const gdn_kv_cache *cache, int32_t n, gdn_dtype dtype, const void *k,
                                 int64_t k_stride_token, int64_t k_stride_head, const void *v,
                                 int64_t v_stride_token, int64_t v_stride_head, const int64_t *slots, void *stream);

/* Softmax attention of one new token per request over its cached tokens:
 *   o[b,h] = sum_j p_j v_j,  p = softmax_j(scale * <q[b,h], k_j>),
 *   lse[b,h] = log sum_j exp(scale * <q[b,h], k_j>)        (lse may be NULL)
 * over the tokens j in [max(0, L - window), L), L = seq_lens[b] (window 0: from
 * 0 on; L is cut at max_pages * page, which is at most 2^31 - 128), whose table entry lies in [0, pages).
 * Query head h reads KV head h / (Hq / Hkv).  A request left without a token
 * gets o = 0 and lse = -inf.  What the cache holds outside those tokens is
 * never used, whatever its bits; a non-finite value inside them reaches only the
 * rows and elements that read it (as infinity or NaN).  In fp32 storage
 * magnitudes from 2^128 - 2^116 up count as infinite.
 * q [B][Hq][d] at b * q_stride_request + h * q_stride_head elements (multiples of
 * 16 bytes); o [B][Hq][d] contiguous; lse [B][Hq] fp32; q and o have the cache's
 * dtype, or GDN_BF16 with a GDN_E4M3 cache.  Row b of the block table starts at
 * b * table_stride (0: all requests share one row, as the rows of a prompt chunk
 * do with seq_lens c+1, c+2, ...).
 * Scores, maxima, sums and outputs are held in fp32.  Weights exp(z - max z) enter
 * the product with V in fewer bits, those of o's type at least: 16 with a GDN_BF16
 * cache; 11 with a GDN_E4M3 one, or 2^-40 of the largest where that is coarser; 22
 * with a GDN_F32 one.  A row's tokens are summed in an order that depends on
 * the lengths of all requests of the call, never on timing: the same call gives
 * the same bits.
 * Workspace: gdn_paged_decode_workspace_bytes(cache, Hq), 256-byte aligned; its
 * contents need no set-up and do not outlive the call.  The call is two launches:
 * host threads that share a stream need a workspace each, as the launches of one
 * may come between those of the other. */
GDN_API size_t gdn_paged_decode_workspace_bytes(const gdn_kv_cache *cache, int32_t Hq);
GDN_API gdn_status gdn_paged_decode(const gdn_kv_cache *cache, int32_t B, int32_t Hq, gdn_dtype dtype, const void *q,
                                    int64_t q_stride_request, int64_t q_stride_head, const int32_t *block_table,
                                    int64_t table_stride, int32_t max_pages, const int32_t *seq_lens, int32_t window,
                                    float scale, void *o, float *lse, void *workspace, size_t workspace_bytes,
                                    void *stream);

/* The next token of every row of logits [B][V] (row b at b * logits_stride
 * elements; GDN_BF16 or GDN_F32; V <= 2^22).  With m the row's largest logit,
 * T = temperature[b], y_i = (x_i - m) / T and w_i = exp(y_i):
 *   K  the top_k[b] largest logits (ties: lowest index first; <= 0 or >= V: all);
 *   P  the shortest prefix of K, in that descending order, whose mass is at least
 *      top_p[b] of K's (>= 1: all of K; at least one token);
 *   the tokens of P with 0 < w_i and w_i >= min_p[b] stay (at least the largest);
 *   tokens[b] = argmax over them of y_i - log(-log u_i), u = noise[b] [V] uniform
 *   random numbers in (0, 1) (clamped to [2^-32, 1 - 2^-24]; ties: lowest index),
 *   which is a draw from the kept weights.
 * logprobs[b] (logprobs may be NULL) = log(w_token / sum_i w_i), over the whole
 * row.  T <= 0: the largest logit (ties: lowest index), logprob 0.  A NULL array
 * stands for T = 1, top_k = 0, top_p = 1, min_p = 0.  Logits of -inf and NaN are
 * never chosen, +inf counts as the largest finite number; a row with neither a
 * finite logit nor +inf gets token -1 and logprob -inf.  The same call gives the
 * same bits: parts of a row are summed in fp32 in a fixed order and joined as
 * 64-bit whole numbers in units of 2^-40 of the largest weight, so that no order of
 * events matters.  The parts depend on B, V and the row's alignment: in another
 * batch a row's logprob may differ in its last bits, and a token at top_p's very
 * edge (within the fp32 rounding of the masses) may fall on its other side.  w_i >= min_p and
 * the scores are fp32 and do not depend on the batch.  No workspace. */
GDN_API gdn_status gdn_sample(int32_t B, int32_t V, gdn_dtype dtype, const void *logits, int64_t logits_stride,
                              const float *noise, int64_t noise_stride, const float *temperature,
                              const int32_t *top_k, const float *top_p, const float *min_p, int32_t *tokens,
                              float *logprobs, void *stream);

/* ---- Prompt chunks through softmax-attention layers -------------------------
 * What a layer does with the new tokens of a step before and after the cache:
 * gdn_qk_rope, then gdn_kv_append of the keys, then gdn_paged_prefill; and
 * gdn_logprobs where a prompt is scored. */

/* Per-head norm and rotary positions of new tokens' queries and keys, in one
 * pass.  Row t, head h of q ([n][Hq][d] at t * q_stride_token + h * q_stride_head
 * elements; k alike with Hkv heads; outputs with strides of their own; all strides
 * multiples of 16 bytes), in fp32 and rounded once:
 *   y = x w / sqrt(mean(x^2) + eps)   with weights [d] fp32 (NULL: y = x);
 *   the first 2 * pairs dims turn by angles positions[t] * freqs[i], i < pairs:
 *   (a, b) -> mscale (a cos - b sin, a sin + b cos) on the pairs (y_i, y_(i+pairs)),
 *   or (y_2i, y_(2i+1)) where `interleaved` is not 0; the other dims stay y.
 * freqs [pairs] fp64 in radians per token (finite); positions any int32.  Angles are
 * products of whole numbers modulo a turn: they lose nothing at far positions beyond
 * what freqs itself, in 53 bits, leaves open.  q_out may be q, and k_out k, with
 * the same strides; apart from that outputs that share memory with q, k, one another or
 * themselves are GDN_ERR_UNSUPPORTED (slices of one projection do not).  d is 64, 128 or 256; Hq or Hkv may be 0, whose
 * pointers are not looked at. */
GDN_API gdn_status gdn_qk_rope(int32_t n, int32_t Hq, int32_t Hkv, int32_t d, gdn_dtype dtype, const void *q,
                               int64_t q_stride_token, int64_t q_stride_head, const void *k, int64_t k_stride_token,
                               int64_t k_stride_head, const int32_t *positions, const double *freqs, int32_t pairs,
                               int32_t interleaved, float mscale, const float *q_weight, const float *k_weight,
                               float eps, void *q_out, int64_t q_out_stride_token, int64_t q_out_stride_head,
                               void *k_out, int64_t k_out_stride_token, int64_t k_out_stride_head, void *stream);

/* Softmax attention of new tokens over the paged cache, which holds them already.
 * Request b's new tokens are the rows cu_new[b] <= t < cu_new[b+1] of q [n][Hq][d]
 * (cut to [0, n]); row t has position p = seq_lens[b] - cu_new[b+1] + t and attends to
 * the tokens j with max(0, p - window + 1) <= j <= p (window 0: from 0 on) and
 * j < max_pages * page, whose table entry lies in [0, pages):
 *   o[t,h] = sum_j p_j v_j,  p = softmax_j(scale * <q[t,h], k_j>),
 *   lse[t,h] = log sum_j exp(scale * <q[t,h], k_j>)           (lse may be NULL).
 * A row left without a token gets o = 0 and lse = -inf.  Rows of no request are not
 * written (a captured step's rows behind cu_new[B]).  o may
 * be q where q is contiguous; apart from that o, lse and the workspace share no memory with
 * one another or an input (GDN_ERR_UNSUPPORTED).
 * Everything else is as in gdn_paged_decode: heads, strides, types, what is never
 * used, where non-finite values reach (a later token's do not reach the rows before it).
 * Weights exp(z - max z) enter the product with V in the bits of o's type or more:
 * 8 with a GDN_BF16 cache; 11 with a GDN_E4M3 one, or 2^-36 of the largest where that
 * is coarser; 22 with a GDN_F32 one.  cu_new does not decrease.  Where it does, nothing
 * but rows of [0, n) that a request names is written: one that several name holds pieces of
 * their attentions, in o and lse apart, and where the requests' rows are more than n in all,
 * some stay as they were.
 * Workspace: gdn_paged_prefill_workspace_bytes(cache, B, n, Hq), 256-byte aligned (41 MB
 * at most, and 76 bytes for every request and every 128 of the n Hq / Hkv rows of a KV head); its contents need no set-up.  The call is several launches: host threads that
 * share a stream need a workspace each, and so do two captured graphs that may run
 * at the same time.  gdn_paged_prefill_status synchronises `stream` and reports
 * the gdn_paged_prefill call that used the workspace last (GDN_ERR_TIMEOUT: a wait
 * inside a kernel ran out and o and lse are not valid); no other kind of call may have
 * used it since.  A call without rows (B or n 0) writes its workspace's status too, where it is
 * given an aligned one. */
GDN_API size_t gdn_paged_prefill_workspace_bytes(const gdn_kv_cache *cache, int32_t B, int32_t n, int32_t Hq);
GDN_API gdn_status gdn_paged_prefill(const gdn_kv_cache *cache, int32_t B, int32_t n, int32_t Hq, gdn_dtype dtype,
                                     const void *q, int64_t q_stride_token, int64_t q_stride_head,
                                     const int32_t *block_table, int64_t table_stride, int32_t max_pages,
                                     const int32_t *seq_lens, const int32_t *cu_new, int32_t window, float scale,
                                     void *o, float *lse, void *workspace, size_t workspace_bytes, void *stream);
GDN_API gdn_status gdn_paged_prefill_status(const void *workspace, void *stream);

/* Self-test of gdn_paged_prefill's failure detection.  With limit_ms of 1 to 2000, in this host thread's
 * following calls, a CTA's copies wait after its first 128 keys for a barrier that nothing arrives at.  The wait runs
 * out after limit_ms, all others end with it, the kernel waits for its copies and products in flight and
 * returns, and the status of a call with more keys is GDN_ERR_TIMEOUT (GDN_F32 caches have no such
 * waits).  0: as normally, where any wait ends after two seconds. */
GDN_API gdn_status gdn_selftest_paged_prefill_wait(int32_t limit_ms);

/* Log probabilities of given tokens, of every row of logits [B][V] (row b at
 * b * logits_stride elements; GDN_BF16 or GDN_F32; V <= 2^30).  With m the row's largest
 * logit and Z = sum_i exp(x_i - m):
 *   logprobs[b] = x_token - m - log Z, token = tokens[b]; 0 for a token outside [0, V);
 *   entropy[b] = log Z - sum_i exp(x_i - m) (x_i - m) / Z          (may be NULL);
 *   top_tokens, top_logprobs [B][top]: the `top` largest logits, descending (ties:
 *   lowest index first), and their log probabilities (top <= 32 and <= V).
 * Logits of -inf have no mass and log probability -inf; among the top they come
 * last.  A row with a NaN or +inf has NaN for every result but top_tokens, where
 * +inf comes first and NaN last; a row of -inf alone has log probabilities of -inf and
 * entropy 0.  Sums are fp32 in a fixed order that depends on B, V and the row's
 * alignment: the same call gives the same bits.  Outputs share no memory with inputs or one another.
 * No workspace. */
GDN_API gdn_status gdn_logprobs(int32_t B, int32_t V, gdn_dtype dtype, const void *logits, int64_t logits_stride,
                                const int32_t *tokens, int32_t top, float *logprobs, float *entropy,
                                int32_t *top_tokens, float *top_logprobs, void *stream);

/* Prefill with HOST inputs and outputs: the same computation as
 * gdn_prefill_sparse (mask != NULL) or gdn_prefill_dense (mask == NULL), with
 * q, k, v, beta, g, h0 (may be NULL), mask and the outputs o, s_final in host
 * memory, laid out as in those calls.  On `stream` the call enqueues one
 * cudaMemcpyAsync per input into device staging carved from the workspace, the
 * prefill, and one cudaMemcpyAsync per output back to the host; it returns
 * without waiting (synchronise the stream before reading o and s_final).  Host
 * buffers should be page-locked (cudaHostAlloc / cudaHostRegister): otherwise
 * the copies do not overlap with other work.  Calls on different streams with
 * different workspaces run concurrently, so a caller can overlap one call's
 * copies with another call's kernels.  Workspace (device, 256-byte aligned):
 * gdn_prefill_host_workspace_bytes(shape, solver, mask != NULL). */
GDN_API gdn_status gdn_prefill_host(const gdn_shape *shape,
                            const void *q, const void *k, const void *v,
                            const float *beta, const float *g, const float *h0,
                            const uint8_t *mask, gdn_solver solver,
                            void *o, float *s_final, void *workspace, size_t workspace_bytes,
                            void *stream);
GDN_API size_t gdn_prefill_host_workspace_bytes(const gdn_shape *shape, gdn_solver solver, int sparse);

/* Allocation-free event-sparse prefill.  The paper has no counterpart: this
 * is a deployment aid for callers that cannot allocate device memory -- for
 * example a plugin inside a host runtime that owns all device memory and
 * passes the plugin only its inputs and outputs, or a latency-critical server
 * that forbids cudaMalloc after start-up.  Same arguments, pipeline and
 * results as gdn_prefill_sparse(), but no workspace argument: the scratch is a
 * fixed array of GDN_NOALLOC_SCRATCH_BYTES (64 MiB) in the library's device
 * memory, which every GPU that loads the library holds until the process
 * exits.  The call allocates nothing and calls no allocating routine.
 *   - Size limit: shapes with gdn_workspace_bytes(shape, solver, 1) above
 *     64 MiB are rejected with GDN_ERR_WORKSPACE before anything is enqueued
 *     (with this version's workspace layout: B=1, Nq=16, bf16 up to
 *     T = 2688; one head pair in fp32 up to T = 20352).
 *   - Set-up: the array belongs to the library's device code, which CUDA loads
 *     lazily: the first call in each context (this entry point or
 *     gdn_noalloc_status) loads it, claiming the 64 MiB then, and looks up its
 *     address with that device current.  Make that first call at start-up,
 *     before a host runtime reserves the rest of the device memory and before
 *     any stream capture.  Every call looks the address up again (no cache), so
 *     a reset context or another context of the same device is handled.
 *   - Sharing: every call uses the same array and it keeps the last call's
 *     contents.  Nothing in it must start at zero (each value read is written
 *     earlier in the same call), but calls that overlap on the GPU (other
 *     streams, other host threads) race on it: serialise them.
 *   - Failure detection: the device status word lives in that array; read it
 *     with gdn_noalloc_status(), which reports the last call on the current
 *     device. */
#define GDN_NOALLOC_SCRATCH_BYTES (64ull << 20)
GDN_API gdn_status gdn_prefill_sparse_noalloc(const gdn_shape *shape,
                                      const void *q, const void *k, const void *v,
                                      const float *beta, const float *g, const float *h0,
                                      const uint8_t *mask, gdn_solver solver,
                                      void *o, float *s_final, float *score, void *stream);

/* Synchronises `stream` and reports the device-latched status (GDN_OK,
 * GDN_ERR_CAPACITY or GDN_ERR_TIMEOUT) of the last gdn_prefill_sparse_noalloc()
 * call on the current device, read from the library's scratch array.  Also
 * loads that array when called first (see the set-up note above).  Allocates
 * nothing.  No counterpart in the paper: part of the allocation-free entry
 * point. */
GDN_API gdn_status gdn_noalloc_status(void *stream);

/* Self-test of failure detection: every wait inside the kernels is bounded in
 * time.  Launches one thread that waits on a barrier nothing arrives at, with
 * a limit of limit_ms (1..2000) milliseconds; the wait must give up, latch the
 * timeout bit (status[2] & 4, the same bit a prefill latches as
 * GDN_ERR_TIMEOUT) and return, leaving the context usable.  status: caller
 * device buffer of 4 int32 (status[3] receives the milliseconds waited).
 * Synchronises `stream`.  Returns GDN_OK when the wait timed out as designed,
 * GDN_ERR_DEVICE when it did not. */
GDN_API gdn_status gdn_selftest_wait_timeout(int32_t *status, int32_t limit_ms, void *stream);

/* Synchronises `stream` and reports the device-latched status of the last
 * prefill that used `workspace` (GDN_OK, GDN_ERR_CAPACITY or GDN_ERR_TIMEOUT). */
GDN_API gdn_status gdn_workspace_status(const void *workspace, void *stream);

GDN_API const char *gdn_status_string(gdn_status status);

/* Stage timing for benchmarks.  enable = 1: each following prefill records a
 * CUDA event before its first and after each pipeline stage on its own stream
 * (stages: 0 compaction, 1 log-decay prefix, 2 intra, 3 deferred W, 4 scan
 * run maps, 5 scan chain over runs, 6 scan (the one-pass scan, the run-map
 * fix-up, or the fp32 scan), 7 group output, 8 online selector; a stage a path
 * does not run reads 0), for up to 256 prefills; while recording, a prefill
 * runs every kernel on the caller's stream, one after another.  enable = 2:
 * nothing is recorded and the prefills keep their normal schedule; only the
 * kernels they launch are counted.  0: off.  Enabling (again) drops earlier
 * records.  Not thread-safe: one host thread drives the profiler.  The events
 * are created on the first enable = 1 (no device memory). */
GDN_API gdn_status gdn_profile_enable(int enable);

/* Synchronises on the recorded events, writes the summed milliseconds of each
 * stage over all recorded prefills to stage_ms[0..n_stages) (n_stages <= 9;
 * zeros under enable = 2), the number of prefills run since enabling to
 * *n_prefills, the number of kernels they launched to *n_launches (may be
 * NULL), and clears the records. */
GDN_API gdn_status gdn_profile_read(float *stage_ms, int32_t n_stages, int32_t *n_prefills,
                                    int64_t *n_launches);

/* Library ABI version (major*10000 + minor*100 + patch). */
GDN_API int32_t gdn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H */
