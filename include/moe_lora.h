/*
 * moe_lora.h -- C ABI of the fused MoE-LoRA expert layer for NVIDIA GB300 (sm_103a).
 *
 * What the layer computes (vLLM blog "multi-LoRA for MoE", vllm.com.cn, section
 * "Implementing multi-LoRA inference for MoE models in vLLM"; and "vLLM Multi-LoRA
 * Serving for MoE Models", agentlenshq.com, section "Multi-LoRA Serving for MoE
 * Models"): each token is routed to its top-k experts; each expert applies a gate_up
 * projection, the gated activation and a down projection, and the experts' outputs
 * are summed with the routing weights. Multi-LoRA adds, per request, a low-rank adapter to both
 * projections: y = xW + (xA)B, where the shrink op is z = xA (h_in -> r) and the
 * expand op is zB (r -> h_out). Token routing and adapter selection together pick
 * an (expert, adapter) pair per token-slot ("compound sparsity").
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - All array pointers are DEVICE pointers owned by the caller. The library never
 *   allocates, frees or synchronises on the compute path; intermediates live in a
 *   caller-provided workspace or align buffer.
 * - Every call is asynchronous on the caller's stream and returns a status code
 *   (moe_lora_status below). Arguments are validated on the host before anything
 *   is launched; on error nothing is launched.
 * - bf16 arrays are passed as `const void*` holding IEEE bfloat16 bit patterns.
 * - Arrays are contiguous and row-major; base pointers of bf16 matrices read by
 *   the tensor-memory-accelerator path must be 16-byte aligned, and their row
 *   length (the reduction dimension) a multiple of 8 elements.
 * - Weight layouts keep the reduction dimension innermost (the transpose of the
 *   pages' h_in x h_out notation, as nn.Linear stores it):
 *       W1 [E, 2I, H]  gate_up (rows [0,I) gate, [I,2I) up)   W2 [E, H, I] down
 *       A1 [L, E, r, H]  B1 [L, E, 2I, r]  A2 [L, E, r, I]  B2 [L, E, H, r]
 *   LoRA scale is 1 (y = xW + xAB); fold any alpha/r into B. Adapters with a
 *   smaller rank are zero-padded to r.
 * - Slots: s = t*k + j for token t and routing choice j. A token's adapter id
 *   -1 means "base model only".
 * - Ids found out of range on the device never trap: the slot is dropped and a
 *   bit is set in a sticky device error word, read back with moe_lora_get_error.
 * - Kernels are chained with programmatic dependent launch on the caller's
 *   stream. Every size is a runtime argument: nothing is compiled or loaded per
 *   token count.
 * - The weights of the layer and of its building blocks (W1, W2, A*, B*) may be
 *   read before earlier launches of the stream have finished, where those trigger
 *   their dependents early, as this library's own kernels do: such launches must
 *   not write them. The feed-forward operators (at the end) read nothing early.
 */
#ifndef MOE_LORA_H_
#define MOE_LORA_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define MOE_LORA_API __attribute__((visibility("default")))
#else
#define MOE_LORA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same underlying type as cudaStream_t; pass a CUDA stream handle (or 0). */
typedef struct CUstream_st* moe_lora_stream_t;

/* Status codes returned by every entry point. */
enum moe_lora_status {
  MOE_LORA_OK = 0,
  MOE_LORA_ERR_INVALID_ARG = 1,          /* null/misaligned pointer, negative size, k > E, ... */
  MOE_LORA_ERR_UNSUPPORTED = 2,          /* shape outside the documented limits, or not an sm_103 device */
  MOE_LORA_ERR_CUDA = 3,                 /* a CUDA runtime call or launch failed */
  MOE_LORA_ERR_WORKSPACE_TOO_SMALL = 4,  /* workspace/align buffer smaller than required */
  MOE_LORA_ERR_TIMEOUT = 5               /* reported by moe_lora_get_error when a bounded wait gave up */
};

/* Bits of the sticky device error word. */
#define MOE_LORA_DEVERR_EXPERT_RANGE 0x1u  /* an expert id outside [0, E): slot dropped */
#define MOE_LORA_DEVERR_ADAPTER_RANGE 0x2u /* an adapter id outside [-1, L): the token's slots dropped */
#define MOE_LORA_DEVERR_TIMEOUT 0x4u       /* a bounded wait inside a kernel gave up; results invalid */
#define MOE_LORA_DEVERR_RANK_RANGE 0x8u    /* an adapter rank outside [0, r]: clamped */

/* Human-readable name of a status code (static string). */
MOE_LORA_API const char* moe_lora_status_string(int status);

/* ---------------------------------------------------------------------------
 * Routing: the router picks each token's top-k experts.
 *
 * moe_topk_softmax: for each of T tokens, ids[t, 0..k) are the indices of the k
 * largest logits[t, :] in decreasing order (equal logits: lower index first; NaN
 * ranks below every number), and w[t, j] = exp(l_j - l_0) / sum_i exp(l_i - l_0)
 * over the chosen logits l_j (fp32). logits [T, E] fp32; ids [T, k] int32;
 * w [T, k] fp32. Requires 1 <= k <= E <= 1024 and k <= 32. T = 0 is a no-op.
 * ------------------------------------------------------------------------- */
MOE_LORA_API int moe_topk_softmax(const float* logits, int T, int E, int k, int32_t* ids, float* w,
                     moe_lora_stream_t stream);

/* ---------------------------------------------------------------------------
 * Alignment: the compound sparsity of expert routing x adapter selection.
 *
 * Slots are stably sorted by the key (expert e, adapter l, slot s), l = -1 first.
 * The result lives in a caller-allocated "align buffer" described by
 * moe_lora_align_t. Its layout (byte offsets from moe_lora_align_layout):
 *   header        int32[64]: [0] error word (uint32, sticky, OR-ed), [1] n_valid,
 *                 [2] n_tiles, [3] n_lora_blocks, [4] n_lora_rows, [5..] echo of
 *                 T, k, E, L, bm_base, bm_lora
 *   sorted_slots  int32[S]    kept slots in key order, -1 after n_valid
 *   slot_row      int32[S]    sorted position of each slot, -1 if dropped
 *   row_expert    int32[S]    expert of each sorted row
 *   row_adapter   int32[S]    adapter of each sorted row (-1: none)
 *   expert_begin  int32[E+1]  rows of expert e are [expert_begin[e], expert_begin[e+1])
 *   tiles         int32[max_tiles][4]  {e, row_begin, rows, 0}: each expert's rows cut
 *                 into chunks of at most bm_base rows (the grouped GEMM's token tiles)
 *   lora_blocks   int32[max_lora_blocks][4] {row_begin, rows, e, l}: each (e, l >= 0)
 *                 segment cut into chunks of at most bm_lora rows
 *   then internal scratch (bucket counts and sort buffers).
 * Entries past the device-side counts are unspecified. Integer results are
 * bit-exact and deterministic.
 * Limits: S = T*k <= 1<<22, E*(L+1)+1 and S together fit 32 key bits,
 * bm_base a multiple of 16 in [16, 256], 1 <= bm_lora <= 16.
 * ------------------------------------------------------------------------- */
typedef struct moe_lora_align_t {
  void* buf;       /* device pointer to an align buffer of moe_lora_align_buffer_size bytes, 256-byte aligned */
  int32_t T;       /* tokens */
  int32_t k;       /* experts per token */
  int32_t E;       /* experts */
  int32_t L;       /* resident adapters (0: none) */
  int32_t bm_base; /* rows per grouped-GEMM token tile */
  int32_t bm_lora; /* rows per LoRA block */
  const int32_t* adapter_ranks; /* optional device array [L]: adapter l has rank r_l in [0, r]
                     and uses only the first r_l rows of each r-row slice of A and the
                     first r_l columns of B (storage stays padded to r); NULL: every
                     adapter has rank r. Used by lora_shrink and lora_expand_add (z
                     entries past r_l are written as 0); 16-byte groups wholly past r_l
                     are never read. Values outside [0, r] are clamped and flagged
                     (MOE_LORA_DEVERR_RANK_RANGE). The pages give one rank per serving
                     instance; per-adapter ranks are this library's extension. */
} moe_lora_align_t;

#define MOE_LORA_ALIGN_NFIELDS 12
/* Indices into the offsets array filled by moe_lora_align_layout. */
enum moe_lora_align_field {
  MOE_LORA_AF_HEADER = 0, MOE_LORA_AF_SORTED_SLOTS, MOE_LORA_AF_SLOT_ROW, MOE_LORA_AF_ROW_EXPERT,
  MOE_LORA_AF_ROW_ADAPTER, MOE_LORA_AF_EXPERT_BEGIN, MOE_LORA_AF_TILES, MOE_LORA_AF_LORA_BLOCKS,
  MOE_LORA_AF_MAX_TILES, MOE_LORA_AF_MAX_LORA_BLOCKS, MOE_LORA_AF_SCRATCH, MOE_LORA_AF_TOTAL_BYTES
};

/* Bytes of align buffer needed; 0 if the parameters are invalid. */
MOE_LORA_API size_t moe_lora_align_buffer_size(int T, int k, int E, int L, int bm_base, int bm_lora);

/* Fills offsets[MOE_LORA_ALIGN_NFIELDS] (byte offsets; MAX_* fields hold counts). Host only. */
MOE_LORA_API int moe_lora_align_layout(int T, int k, int E, int L, int bm_base, int bm_lora, int64_t* offsets);

/* ids [T, k] int32; token_adapter [T] int32 or NULL (all -1). Deterministic. Below 2048
 * slots (or with more buckets E*(L+1)+1 than half the slots) one CTA sorts every slot;
 * from 2048 slots three launches share the work: per-CTA stable sorts of 512-slot chunks,
 * one scan over the (key, chunk) count table, and a placement pass. */
MOE_LORA_API int moe_lora_align(const int32_t* ids, const int32_t* token_adapter, const moe_lora_align_t* al,
                   moe_lora_stream_t stream);

/* Copies the sticky error word of an align buffer (or of a layer workspace, whose
 * first bytes are its align buffer) to *err. Synchronises `stream`. */
MOE_LORA_API int moe_lora_get_error(const void* align_buf_or_workspace, moe_lora_stream_t stream, uint32_t* err);
/* Clears the sticky error word (asynchronous). */
MOE_LORA_API int moe_lora_clear_error(void* align_buf_or_workspace, moe_lora_stream_t stream);

/* ---------------------------------------------------------------------------
 * Gather: xs[row, :] = x[sorted_slots[row] / k, :] for the n_valid sorted rows.
 * x [T, H] bf16; xs [S, H] bf16 (rows past n_valid untouched).
 * ------------------------------------------------------------------------- */
MOE_LORA_API int moe_gather_rows(const void* x, const moe_lora_align_t* al, int H, void* xs,
                    moe_lora_stream_t stream);

/* ---------------------------------------------------------------------------
 * Base expert grouped GEMM (vLLM's fused_moe group GEMM, one GEMM per expert
 * over the tokens routed to it; vllm.com.cn, section "Implementing multi-LoRA
 * inference for MoE models in vLLM").
 *   out[row, n] = sum_c a[row, c] * W[e(row), n, c]   for row < n_valid
 * a [S, K] bf16 in sorted-row order; W [E, N, K] bf16; out [S, N] fp32 (rows past
 * n_valid untouched). bf16 in, fp32 accumulate on the tcgen05 tensor cores with
 * TMEM accumulators, operands staged by TMA. Requires K % 8 == 0, 16-byte aligned
 * a and W, N >= 1.
 * ------------------------------------------------------------------------- */
MOE_LORA_API int moe_grouped_gemm(const void* a, const void* W, const moe_lora_align_t* al, int N, int K,
                     float* out, moe_lora_stream_t stream);

/* ---------------------------------------------------------------------------
 * LoRA shrink z = xA for every slot whose token has an adapter (vllm.com.cn,
 * sections "Implementing ..." and "Kernel optimizations": r outputs, each a long
 * sum over h_in, so the sum over K is split across warps of a CTA).
 *   Z[s, i] = sum_c X[in(s), c] * A[l(s), e(s), i, c]
 * rows_are_slots = 0: in(s) = s / k, X is [T, K] (token activations).
 * rows_are_slots = 1: in(s) = slot_row[s], X is [S, K] (sorted rows, e.g. the
 *                     SwiGLU output feeding the down projection).
 * A [L, E, r, K] bf16; Z [S, r] fp32 (slots without adapter untouched).
 * With al->adapter_ranks, adapter l uses rows [0, r_l) of A and Z[s, i >= r_l] = 0.
 * Any K >= 1 and 1 <= r <= 256; K % 8 == 0 with 16-byte aligned X and A takes the
 * 128-bit load path, and K % 32 == 0 also drops the bounds masks (EVEN_K).
 * Deterministic (fixed-order reductions, no atomics).
 * ------------------------------------------------------------------------- */
MOE_LORA_API int lora_shrink(const void* X, int rows_are_slots, const void* A, const moe_lora_align_t* al,
                int K, int r, float* Z, moe_lora_stream_t stream);

/* ---------------------------------------------------------------------------
 * LoRA expand with the base add fused in (vllm.com.cn, section "Kernel
 * optimizations": the LoRA result is added to the base output inside the expand
 * kernel), plus the layer's epilogues:
 *   delta[row, n] = sum_i Z[s, i] * B[l, e, n, i]      (rows with an adapter)
 *   epilogue 0: base[row, n] += delta[row, n]           in place, fp32 [S, N]
 *   epilogue 1: out[row, n] = silu(g) * u with g = base[row, n] + delta[row, n],
 *               u = base[row, N/2 + n] + delta[row, N/2 + n]; out [S, N/2] bf16,
 *               every valid row (with or without adapter). N must be even.
 *   epilogue 2: out[t, n] = sum_j w[t, j] * (base[row(t,j), n] + delta[row(t,j), n]),
 *               j in increasing order; out [T, N] bf16 (out_fp32 = 0) or fp32.
 *               base is only read.
 *   epilogue 3: as epilogue 1 with separate gate and up adapters: Z rows hold 2r
 *               values, columns [0, N/2) take z[0, r) and B rows [0, N/2), columns
 *               [N/2, N) take z[r, 2r) and B rows [N/2, N); B stays [L, E, N, r].
 * Z [S, r] fp32 ([S, 2r] for epilogue 3); B [L, E, N, r] bf16 (NULL or L = 0: no
 * adapter term). With al->adapter_ranks, adapter l uses columns [0, r_l) of B only.
 * topk_w [T, k] fp32 (epilogue 2 only). Requires L < 65535. Deterministic.
 * ------------------------------------------------------------------------- */
MOE_LORA_API int lora_expand_add(const float* Z, const void* B, const moe_lora_align_t* al, int N, int r,
                    int epilogue, float* base, void* out, int out_fp32, const float* topk_w,
                    moe_lora_stream_t stream);

/* ---------------------------------------------------------------------------
 * The whole layer, as one of two chains of launches (moe_lora_layer_plan says which):
 *   route (if logits != NULL) -> align -> gather -> gate_up grouped GEMM ->
 *   gate_up shrink -> gate_up expand + SwiGLU -> down grouped GEMM -> down shrink
 *   -> down expand + weighted top-k combine;
 * or, with the expand fused into the grouped GEMMs by concatenation along K
 * (y = xW + zB = [x | z][W | B]^T for the rows of each adapter):
 *   route -> align -> gather -> gate_up shrink -> gate_up GEMM + expand + SwiGLU ->
 *   down shrink -> down GEMM + expand -> weighted top-k combine.
 * x [T, H] bf16. Routing: either logits [T, E] fp32 (topk_ids/topk_w NULL) or
 * caller-provided topk_ids [T, k] int32 and topk_w [T, k] fp32 (logits NULL).
 * token_adapter [T] int32 or NULL. LoRA weights may be NULL with L = 0 (base MoE).
 * y [T, H]: bf16 (y_fp32 = 0) or fp32. workspace: moe_lora_workspace_size bytes,
 * 256-byte aligned; its first bytes are the layer's align buffer (error word).
 * Requires H % 8 == 0, I % 8 == 0, 1 <= k <= min(E, 32), E <= 1024, L < 65535.
 * ------------------------------------------------------------------------- */
MOE_LORA_API size_t moe_lora_workspace_size(int T, int k, int E, int L, int H, int I, int r);

MOE_LORA_API int moe_lora_layer(const void* x, const float* logits, const int32_t* topk_ids,
                   const float* topk_w, const int32_t* token_adapter, int T, int H, int I, int E,
                   int k, const void* W1, const void* W2, const void* A1, const void* B1,
                   const void* A2, const void* B2, int L, int r, void* y, int y_fp32,
                   void* workspace, size_t workspace_bytes, moe_lora_stream_t stream);

/* Optional controls for moe_lora_layer_ex (zero-initialise, then set fields). */
typedef struct moe_lora_layer_opts {
  int32_t bm_base;      /* grouped-GEMM token tile; 0 = heuristic */
  int32_t bm_lora;      /* LoRA block rows; 0 = heuristic */
  int32_t disable_pdl;  /* 1: plain stream-ordered launches */
  int32_t num_events;   /* length of `events` (0: none) */
  void** events;        /* cudaEvent_t handles recorded on `stream` before each stage and
                           after the last: [0] route, [1] align (at few tokens the align
                           routes them itself: [0] and [1] mark the same point), [2]
                           gather, then for the
                           chain with a separate expand: [3] gate_up GEMM, [4] gate_up
                           shrink, [5] gate_up expand+SwiGLU, [6] down GEMM, [7] down shrink,
                           [8] down expand+combine; for the fused chain
                           (moe_lora_layer_plan_t.fused_expand): [3] gate_up shrink, [4]
                           gate_up GEMM with expand+SwiGLU, [5] empty, [6] down shrink, [7]
                           down GEMM with expand, [8] combine; [9] end */
  const int32_t* adapter_ranks; /* optional device array [L] of per-adapter ranks (see
                           moe_lora_align_t.adapter_ranks); NULL: every adapter has rank r */
  int32_t gate_up_slices; /* 0 or 1: one adapter over the fused gate_up output (A1
                           [L,E,r,H]); 2: separate gate and up adapters, A1 [L,E,2r,H]
                           with the gate A in rows [0,r) and the up A in [r,2r), B1
                           [L,E,2I,r] unchanged: gate columns take the gate z, up columns
                           the up z (lora_expand_add epilogue 3). The pages describe one
                           adapter per projection and are silent on a split gate_up. */
  int32_t expand_mode;  /* 0: the library picks; 1: the expand in kernels of its own (after
                           each grouped GEMM); 2: the fused chain (the expand as extra K-steps
                           of the grouped GEMMs, SwiGLU in the gate_up GEMM's epilogue)
                           wherever it applies: one adapter rank (no adapter_ranks), one
                           gate_up slice, r % 8 == 0, and shapes whose shifted z buffers stay
                           small (they grow with E * L). The library picks the fused chain
                           where it applies and pays: with adapters, at few rows per expert or
                           at (expert, adapter) runs of 16 rows or more on average; without,
                           with token tiles. Both chains compute the same function; their
                           results differ in fp32 summation order only. */
  int64_t wait_limit_ns; /* for tests of the give-up path: the wall-time limit of the grouped
                           GEMMs' main-loop mbarrier waits (and of the short-K shrink's slab
                           wait). 0: the default, 4 s; < 0: give up at the first unsuccessful
                           poll. A wait that gives up sets MOE_LORA_DEVERR_TIMEOUT; the CTA then
                           drains its own copies and tensor-core work (those waits keep the 4 s
                           limit), frees its tensor memory and exits, and that launch's
                           results are invalid. */
  int32_t mma_pairs;    /* fused chain with 256-row token tiles: 0 = the library's choice
                           (pairs of CTAs, each job one tcgen05.mma.cta_group::2 of M = 256
                           over two 128-row weight blocks, each CTA staging half the token
                           rows); -1 = one CTA per 128-row weight block. Same results up to
                           fp32 summation order. */
} moe_lora_layer_opts;

#define MOE_LORA_LAYER_NUM_STAGES 9

MOE_LORA_API int moe_lora_layer_ex(const void* x, const float* logits, const int32_t* topk_ids,
                      const float* topk_w, const int32_t* token_adapter, int T, int H, int I,
                      int E, int k, const void* W1, const void* W2, const void* A1,
                      const void* B1, const void* A2, const void* B2, int L, int r, void* y,
                      int y_fp32, void* workspace, size_t workspace_bytes,
                      const moe_lora_layer_opts* opts, moe_lora_stream_t stream);

/* ---------------------------------------------------------------------------
 * One serving step with its per-step inputs and its output in host memory: the
 * same layer as moe_lora_layer_ex, routed from logits, with the copies in and out
 * issued by the library on the same stream. The pages describe the device-side
 * computation only; this call stages it for a caller whose batch arrives in host
 * memory (the router logits and adapter ids of a decode step, for instance).
 *
 * moe_lora_host_io_layout (host only) gives the byte offsets, each 256-byte aligned:
 *   offsets[0] x [T, H] bf16, offsets[1] logits [T, E] fp32,
 *   offsets[2] token_adapter [T] int32 (with_adapter = 1; else -1),
 *   offsets[3] y [T, H] bf16 (y_fp32 = 0) or fp32.
 * The caller's host input block holds x, logits and (with_adapter) the adapter ids
 * at offsets[0..2] and is *in_bytes long; the device staging area, *staging_bytes
 * long, holds the same inputs plus y at offsets[3].
 *
 * moe_lora_layer_host enqueues on `stream`, in order: one cudaMemcpyAsync of the
 * whole input block (in_bytes) into `staging`; the layer on the staged views
 * (moe_lora_layer_ex with logits routing; token_adapter NULL when with_adapter = 0;
 * weights, workspace and opts as there); one cudaMemcpyAsync of y into y_host
 * (T*H*2 bytes, or T*H*4 with y_fp32). It returns without waiting: synchronise the
 * stream before reading y_host or rewriting in_host. Page-locked host memory keeps
 * both copies asynchronous; pageable memory works but the copies then synchronise
 * with the host. staging: device memory, 256-byte aligned, at least staging_bytes.
 * Errors: every argument, the layer's included, is checked before anything is
 * copied or launched (MOE_LORA_ERR_WORKSPACE_TOO_SMALL for a short staging area).
 * ------------------------------------------------------------------------- */
MOE_LORA_API int moe_lora_host_io_layout(int T, int H, int E, int with_adapter, int y_fp32,
                                         int64_t* offsets, size_t* in_bytes,
                                         size_t* staging_bytes);

MOE_LORA_API int moe_lora_layer_host(const void* in_host, void* y_host, void* staging,
                                     size_t staging_bytes, int with_adapter, int T, int H, int I,
                                     int E, int k, const void* W1, const void* W2, const void* A1,
                                     const void* B1, const void* A2, const void* B2, int L, int r,
                                     int y_fp32, void* workspace, size_t workspace_bytes,
                                     const moe_lora_layer_opts* opts, moe_lora_stream_t stream);

/* Tile sizes the layer picks for a shape (host only): bm_base, bm_lora. */
MOE_LORA_API int moe_lora_layer_tiles(int T, int k, int E, int L, int H, int I, int r, int32_t* bm_base,
                         int32_t* bm_lora);

/* How moe_lora_layer_ex runs a shape with the given options (NULL: defaults); host only.
 *   bm_base, bm_lora      the align's token tile and LoRA block rows
 *   expert_major_rows     > 0: each grouped-GEMM CTA takes one (expert, 128-row weight block)
 *                         and all of the expert's rows in chunks of this many (few rows per
 *                         expert); 0: token tiles of bm_base rows
 *   fused_expand          1: the LoRA expand runs as extra K-steps of the grouped GEMMs
 *                         (y = [x | z][W | B]^T per adapter run of a tile; the gate_up GEMM
 *                         writes the SwiGLU output directly, the down GEMM its rows, then a
 *                         combine kernel); 0: the expand in kernels of its own
 *   launches              kernels one call launches when routed from logits (one fewer with
 *                         caller-provided ids)
 *   early_reads           (kernel, earlier step) pairs where a kernel reads that step's
 *                         output before its own griddepcontrol.wait (programmatic dependent
 *                         launch). The plan checks each: the producer is at least two launches
 *                         back and the launch in between triggers its dependents only after its
 *                         own wait, so the producer has completed when the reader starts; a
 *                         chain that broke this would be refused (MOE_LORA_ERR_UNSUPPORTED).
 *   route_in_align        1: routed from logits, the one-CTA align routes the tokens itself
 *                         (up to 64 tokens, 64 experts): no separate route launch */
typedef struct moe_lora_layer_plan_t {
  int32_t bm_base;
  int32_t bm_lora;
  int32_t expert_major_rows;
  int32_t fused_expand;
  int32_t launches;
  int32_t early_reads;
  int32_t route_in_align;
} moe_lora_layer_plan_t;

MOE_LORA_API int moe_lora_layer_plan(int T, int k, int E, int L, int H, int I, int r,
                                     const moe_lora_layer_opts* opts, moe_lora_layer_plan_t* plan);

/* ---------------------------------------------------------------------------
 * moe_lora_layer_noalloc: the same layer as moe_lora_layer for callers that cannot
 * allocate device memory -- e.g. a serving engine that has reserved nearly all HBM
 * for weights and KV cache and hands out only its own buffers, a plugin interface
 * that passes inputs and outputs but no allocator, or a latency-critical path
 * where cudaMalloc/cudaFree may synchronise the device. The pages describe no such
 * entry point; it has no counterpart there.
 * Arguments are moe_lora_layer's without the workspace; intermediates live in a
 * 64 MiB array in device global memory held by the library (every GPU that loads
 * it keeps the 64 MiB until the process exits). Shapes whose
 * moe_lora_workspace_size exceeds 64 MiB return MOE_LORA_ERR_WORKSPACE_TOO_SMALL
 * and launch nothing. err_out: optional device pointer that receives this call's
 * device error word (MOE_LORA_DEVERR_* bits; cleared at the start of each call).
 * The function allocates nothing. All calls on a device share the array and it
 * keeps the last call's contents: calls that overlap on the GPU race, so order
 * them on one stream. The first call on each device looks up the array's device
 * address; make that first call before any stream capture. The address belongs to
 * the device's current context: after that context is re-created (cudaDeviceReset)
 * the next call looks it up again.
 * ------------------------------------------------------------------------- */
MOE_LORA_API int moe_lora_layer_noalloc(const void* x, const float* logits,
                                        const int32_t* topk_ids, const float* topk_w,
                                        const int32_t* token_adapter, int T, int H, int I, int E,
                                        int k, const void* W1, const void* W2, const void* A1,
                                        const void* B1, const void* A2, const void* B2, int L,
                                        int r, void* y, int y_fp32, uint32_t* err_out,
                                        moe_lora_stream_t stream);

/* ---------------------------------------------------------------------------
 * The feed-forward block by itself: training in 16 bits, gradient clipping, and
 * 4-bit weights for serving. Element types and activations:
 * ------------------------------------------------------------------------- */
enum moe_dtype { MOE_DTYPE_BF16 = 0, MOE_DTYPE_FP16 = 1, MOE_DTYPE_FP32 = 2 };
enum moe_act {
  MOE_ACT_NONE = 0,
  MOE_ACT_SILU = 1, /* a(g) = g / (1 + exp(-g)) */
  MOE_ACT_GELU = 2  /* a(g) = g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) / 2 */
};

/* Sticky device error word of moe_gated_ffn and its backward, which have no align buffer to
 * keep one in: MOE_LORA_DEVERR_* bits raised on the current device since it was last
 * cleared. The first waits for the stream. Either's first call in a context, and the first
 * moe_gated_ffn, looks the word's address up: make it before a stream capture. */
MOE_LORA_API int moe_ffn_get_error(moe_lora_stream_t stream, uint32_t* err);
MOE_LORA_API int moe_ffn_clear_error(moe_lora_stream_t stream);
/* For tests of the give-up paths: the wall-time limit, in ns, of the main waits of these kernels
 * in the calling thread's later calls. 0: the default (4 s); negative: give up at the first
 * unsuccessful poll. */
MOE_LORA_API int moe_ffn_set_wait_limit(int64_t ns);

/* ---------------------------------------------------------------------------
 * moe_gated_ffn: h[t, i] = a(g) * u with g = x[t] . W1[i] and u = x[t] . W1[I + i].
 * x [T, H], W1 [2I, H] (rows [0, I) gate, [I, 2I) up), h [T, I], all of `dtype`
 * (bf16 or fp16). g and u are summed and the activation evaluated in fp32; h is rounded
 * once. T = 0 is a no-op. H and I are multiples of 8, the pointers 16-byte aligned. Nothing is
 * read before every earlier launch of the stream is over: x and W1 may be their outputs.
 * ------------------------------------------------------------------------- */
MOE_LORA_API int moe_gated_ffn(const void* x, const void* W1, int dtype, int act, int T, int H,
                               int I, void* h, moe_lora_stream_t stream);

/* ---------------------------------------------------------------------------
 * moe_gated_ffn_backward: the gradients of moe_gated_ffn for dh [T, I]. With g and u
 * computed again from x and W1 in fp32,
 *   dg = dh * u * a'(g),  du = dh * a(g)      (rounded once to `dtype`: the tensor cores'
 *                                              operand type),
 *   dx = dg Wg + du Wu  [T, H],   dW1 = [dg^T x ; du^T x]  [2I, H],
 * summed in fp32 and rounded once. dx or dW1 may be null (not wanted). T = 0 writes a
 * zero dW1. The workspace holds dg and du: moe_gated_ffn_backward_workspace_size bytes,
 * 256-byte aligned (0: shape not supported); it needs no initialisation. The sums' order is
 * fixed: results do not vary from run to run.
 * ------------------------------------------------------------------------- */
MOE_LORA_API size_t moe_gated_ffn_backward_workspace_size(int T, int H, int I);
MOE_LORA_API int moe_gated_ffn_backward(const void* dh, const void* x, const void* W1, int dtype,
                                        int act, int T, int H, int I, void* dx, void* dW1,
                                        void* workspace, size_t workspace_bytes,
                                        moe_lora_stream_t stream);

/* ---------------------------------------------------------------------------
 * moe_grad_clip: norm = sqrt(sum of squares over all n tensors) and, with outs,
 * outs[i] = grads[i] * min(1, max_norm / (norm + 1e-6)), rounded to the tensor's type.
 * grads, outs, numels and dtypes are HOST arrays of n entries (device pointers, element
 * counts >= 0, moe_dtype values), read before the call returns; outs may be null (the norm
 * only), and outs[i] may equal grads[i] (in place) but may not overlap any other tensor.
 * Tensors are contiguous and aligned to their element; a pair whose addresses differ modulo
 * 16 bytes is stored element by element. norm: fp32 on the device. Squares are
 * summed in fp32 within a CTA (carrying the rounding along from chunk to chunk, then in a
 * tree) and in fp64 from there on; squares past fp32's range give an infinite norm and a NaN
 * anywhere a NaN norm; both scale as the formula says (zeros, and NaN where a gradient is not
 * finite; NaN everywhere). max_norm >= 0; infinity scales nothing, whatever the norm. The
 * workspace holds partial sums:
 * moe_grad_clip_workspace_size bytes, 16-byte aligned, needs no initialisation. The sum's
 * order is fixed by the sizes and alignments: results do not vary from run to run.
 * ------------------------------------------------------------------------- */
MOE_LORA_API size_t moe_grad_clip_workspace_size(int n, const int64_t* numels);
MOE_LORA_API int moe_grad_clip(const void* const* grads, void* const* outs, const int64_t* numels,
                               const int32_t* dtypes, int n, float max_norm, float* norm,
                               void* workspace, size_t workspace_bytes, moe_lora_stream_t stream);

/* ---------------------------------------------------------------------------
 * 4-bit weights. Natural form: codes [E, N, ceil(K/2)] uint8, code of column 2j in the low
 * half of byte j; scales [E, N, ceil(K/group)] of `dtype` (bf16 or fp16); zeros [E, N,
 * ceil(K/group)] uint8 in 0..15, or null for 8 everywhere. Weight n, c of expert e is
 *   (codes[e, n, c] - zeros[e, n, c / group]) * scales[e, n, c / group].
 * group is 32, 64 or 128.
 *
 * moe_w4_quantize makes codes and scales of W [E, N, K] (bf16 or fp16, finite; zeros 8): the
 * scale of a group is its largest magnitude / 7, rounded to `dtype`, and a code is the
 * nearest of the 15 levels -7..7 plus 8, ties to even. (A group of zeros: scale 0, codes 8.)
 *
 * moe_w4_pack lays the natural form out for moe_w4_matvec, once per weight: rows in tiles
 * of 16, columns in chunks of 128, each (tile, chunk) 1 KiB in the order the lanes of a warp
 * read it; then the scales and the zeros in the same order. `gated`: the rows [0, N/2) and
 * [N/2, N) are tiled by themselves, as the gated form needs (N even). packed:
 * moe_w4_packed_size bytes, 16-byte aligned. K is a multiple of 8 and at most 16384, as the product
 * takes it: other weights are refused here.
 * ------------------------------------------------------------------------- */
MOE_LORA_API int moe_w4_quantize(const void* W, int dtype, int E, int N, int K, int group,
                                 uint8_t* codes, void* scales, moe_lora_stream_t stream);
MOE_LORA_API size_t moe_w4_packed_size(int E, int N, int K, int group, int has_zeros, int gated);
MOE_LORA_API int moe_w4_pack(const uint8_t* codes, const void* scales, const uint8_t* zeros, int E,
                             int N, int K, int group, int gated, void* packed,
                             moe_lora_stream_t stream);

enum { MOE_W4_ROWS_SORTED = 1, MOE_W4_ZERO_DROPPED = 2 };

/* moe_w4_matvec: out[i, n] = x[row(i)] . W[e(i), n] for few rows. A weight is read once per pass
 * over its expert's rows, as many as fit into shared memory: 32 up to K = 2688, 16 up to 5504, 8 up
 * to 11136, 6 at 14336; in the gated form 16 up to K = 4096, 8 up to 8192, 4 at 14336; and at most
 * 8 where the experts get 4 rows or fewer on average. Sums are fp32, and every code - zero
 * enters them exactly; a group's sum is scaled in fp32. Infinities and NaN in x meet code - zero as
 * a product does (0 times infinity: NaN), and stay in their row. `dtype` is the type of x and of
 * the scales.
 *   al null: E = 1, R = T rows, row(i) = i.
 *   al given (al->E = E, al->T = T): the rows of moe_lora_align's sorted order, R = T * al->k;
 *     row_flags = 0: x [T, K] holds tokens, row(i) = sorted_slots[i] / k;
 *     MOE_W4_ROWS_SORTED: x [R, K] is in sorted order (a previous product's output).
 *     Rows of dropped slots are not written, or with MOE_W4_ZERO_DROPPED set to zero.
 * act MOE_ACT_NONE: out [R, N], fp32 (out_fp32 = 1; what lora_expand_add takes as its base)
 * or `dtype`. With an activation the packing must be gated and out [R, N/2] of `dtype` is
 * a(gate) * up. K is a multiple of 8 and at most 16384, x 16-byte aligned. T = 0 is a no-op. */
MOE_LORA_API int moe_w4_matvec(const void* x, int dtype, const void* packed, int E, int N, int K,
                               int group, int has_zeros, int gated, int act, int T,
                               const moe_lora_align_t* al, int row_flags, void* out,
                               int out_fp32, moe_lora_stream_t stream);

/* ---------------------------------------------------------------------------
 * Around the experts' products: rows by expert and back, the router's gradient, and a
 * projection with the adapters of many requests, each with its gradient. The rows are those of
 * moe_lora_align; a buffer that gave a forward pass its order gives the backward pass the same
 * order, so it must not be aligned anew in between. `dtype` is the type of the rows. Nothing
 * is read before every earlier launch of the stream is over. No atomics: results do not vary
 * from run to run.
 * ------------------------------------------------------------------------- */
enum {
  MOE_ROWS_SORTED = 1,      /* the operands' rows are in sorted order (else: row s is slot s) */
  MOE_ROWS_ZERO_DROPPED = 2 /* output rows that no kept slot writes are set to zero (else: left) */
};

/* moe_permute: xs[row] = x[sorted_slots[row] / k] for the n_valid sorted rows; x [T, H], xs
 * [S, H] (bf16, fp16 or fp32). Without MOE_ROWS_ZERO_DROPPED, rows past n_valid are left.
 * moe_unpermute: y[t] = sum over j of w[t, j] o[slot_row[t, j]], j ascending, in fp32 and rounded
 * once; o [S, H], y [T, H], w [T, k] fp32 or null for ones. Dropped slots add nothing, whatever
 * their weight; a token without a kept slot gets zeros. With w null it is moe_permute's gradient,
 * and moe_unpermute_backward with w and dw null is its own.
 * moe_unpermute_backward: d_o[slot_row[t, j]] = w[t, j] dy[t], rounded once, and dw[t, j] =
 * <o[slot_row[t, j]], dy[t]> summed in fp32 (0 for a dropped slot). d_o or dw may be null (not
 * wanted); o is read for dw only. Outputs overlap no input. Any H up to 2^24; pointers aligned
 * to their element (16-byte alignment and rows of a multiple of 16 bytes are fastest). */
MOE_LORA_API int moe_permute(const void* x, int dtype, const moe_lora_align_t* al, int H, int row_flags,
                             void* xs, moe_lora_stream_t stream);
MOE_LORA_API int moe_unpermute(const void* o, int dtype, const moe_lora_align_t* al, const float* w, int H,
                               void* y, moe_lora_stream_t stream);
MOE_LORA_API int moe_unpermute_backward(const void* dy, const void* o, int dtype, const moe_lora_align_t* al,
                                        const float* w, int H, int row_flags, void* d_o, float* dw,
                                        moe_lora_stream_t stream);

/* moe_topk_softmax_backward: the gradient of moe_topk_softmax's weights with respect to the
 * logits: dlogits[t, ids[t, j]] = w_j (dw_j - sum over i of w_i dw_i), zero for experts not
 * chosen. dw, w [T, k] and dlogits [T, E] fp32, ids [T, k] int32; ids outside [0, E) take no
 * part, and equal ids of a token add up. Limits as moe_topk_softmax. */
MOE_LORA_API int moe_topk_softmax_backward(const float* dw, const int32_t* ids, const float* w, int T, int E,
                                           int k, float* dlogits, moe_lora_stream_t stream);

/* ---------------------------------------------------------------------------
 * moe_lora_linear: a projection with low-rank adapters beside it. For every kept row, of
 * expert e and adapter l (-1: none),
 *   z = x A[l, e]^T (fp32),   y = x W[e]^T + z B[l, e]^T,   rounded once.
 * W [E, N, K], A [L, E, r, K], B [L, E, N, r], all of `dtype` (bf16 or fp16). E = 1 is one
 * projection shared by every row. With MOE_ROWS_SORTED x [S, K] and y [S, N] are in sorted order
 * (moe_permute's); else k = 1 and row t is token t. Sums are fp32; z enters the second
 * product as two values of `dtype` (its rounding and the remainder's): off by 2^-17 of it at most in
 * bf16, in fp16 by 2^-23 of it or 2^-25, whichever is more (2^-25 below 1/4: a small z against weights far
 * above 1 shows it). A z that is infinite in `dtype` (in fp16 past 65504) is infinite. No row meets another
 * adapter's weights: an infinity or NaN in them stays with their own rows (where an infinite weight
 * of B gives infinity or NaN).
 *
 * moe_lora_linear_backward: for dy, with z and v = dy B[l, e] in fp32,
 *   dx = dy W[e] + v A[l, e],   dA[l, e] = v^T x,   dB[l, e] = dy^T z
 * over each adapter's rows, rounded once; dA and dB are written for every (adapter, expert)
 * pair, zero where it has no row. v enters dx as z does y; z and v enter dA and dB likewise (in fp16 off by
 * 2^-23 of them or 2^-36).
 * W is frozen: it has no gradient. dx, dA or dB may be null (not wanted).
 *
 * The align buffer needs L >= 1 and no adapter_ranks; bm_base 256 and bm_lora 16 are fastest. N, K
 * and r are multiples of 8, r at most 128, E L at most 2^20, N K below 2^39, and the tiles of 64 columns
 * below 2^30; pointers are 16-byte aligned; outputs overlap no input. workspace: moe_lora_linear_workspace_size bytes (0: not supported; al->buf is
 * not looked at), 256-byte aligned, needs no initialisation. A wait that gives up sets the word of moe_ffn_get_error.
 * Up to 128 rows of one expert the sums' order differs from that for more.
 * ------------------------------------------------------------------------- */
MOE_LORA_API size_t moe_lora_linear_workspace_size(const moe_lora_align_t* al, int N, int K, int r,
                                                   int row_flags, int backward);
MOE_LORA_API int moe_lora_linear(const void* x, const void* W, const void* A, const void* B, int dtype,
                                 const moe_lora_align_t* al, int N, int K, int r, int row_flags, void* y,
                                 void* workspace, size_t workspace_bytes, moe_lora_stream_t stream);
MOE_LORA_API int moe_lora_linear_backward(const void* dy, const void* x, const void* W, const void* A,
                                          const void* B, int dtype, const moe_lora_align_t* al, int N, int K,
                                          int r, int row_flags, void* dx, void* dA, void* dB, void* workspace,
                                          size_t workspace_bytes, moe_lora_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_LORA_H_ */
