/*
 * fdllm.h - C ABI of the Flash-dLLM per-layer hot path on NVIDIA B200 (sm_100a).
 *
 * One layer step of masked-diffusion decoding with Flash-dLLM KV caching:
 *   (a) Flash-Cache: the selected rows' hidden states go through the QKV
 *       projection, RoPE is applied, and K/V are written from on-chip memory
 *       straight into a paged KV cache; Q never leaves the SM.
 *   (b) scheduled attention: each sequence's query rows attend over that
 *       sequence's pages through its block table, so one launch covers a
 *       batch whose sequences differ in length and in stage; the Flash-Verify
 *       two-view mask is applied inside the same kernel, and each key's
 *       accumulated attention mass is emitted for the next step's top-k
 *       tracking set.
 *
 * Sources (cited by page title and paragraph):
 *   [FD] "Flash-dLLM: I/O-Aware KV Caching and Parallel Decoding for Fast,
 *        Memory-Efficient Diffusion LLMs" (ai4snews summary of the full text).
 *        Paragraph 1: Flash-Cache fuses QKV projection, RoPE and the cache
 *        write; scheduled Flash Attention aligns query blocks with their KV
 *        blocks through a block table across caching and update stages.
 *        Paragraph 2: each step's queries are a sliding unmasking window plus
 *        a fixed tracking budget of most-attended tokens.
 *        Paragraph 3: Flash-Verify places a draft view and a mask view at the
 *        same positions, sharing positional embeddings, isolated from each
 *        other by a causal mask inside the fused kernel.
 *   [AB] "Flash-dLLM: IO-Aware KV Caching and Parallel Decoding for Fast,
 *        Memory-Efficient Diffusion LLMs" (arXiv abstract page), Abstract:
 *        GPU memory I/O is the dominant bottleneck; an I/O-aware fused
 *        KV-cache kernel reduces redundant memory movement.
 *
 * Conventions for every entry point:
 *   - Pointers documented DEVICE are CUDA device pointers owned by the
 *     caller and borrowed for the duration of the call (and of the work it
 *     enqueues). Pointers documented HOST are read before the call returns.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream). Work is enqueued asynchronously; nothing synchronises except
 *     fdllm_check, fdllm_cache_create and steps run with validate = 1.
 *   - Host-detectable errors return a status and enqueue nothing.
 *     fdllm_last_error() returns a message for the calling thread.
 *   - Device-detected errors (a page id outside the pool, a slot past the
 *     block table, a position outside the RoPE table) skip the offending
 *     row, never trap, and are reported by the next fdllm_check as
 *     FDLLM_ERR_DEVICE_BOUNDS.
 *   - The library is single-GPU: every pointer must live on the device that
 *     was current at fdllm_cache_create.
 */
#ifndef FDLLM_H
#define FDLLM_H

#include <stdint.h>

#if defined(__GNUC__)
#define FDLLM_API __attribute__((visibility("default")))
#else
#define FDLLM_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FDLLM_OK = 0,
  FDLLM_ERR_INVALID_ARG = 1,   /* bad pointer, size or shape (host check) */
  FDLLM_ERR_UNSUPPORTED = 2,   /* valid request outside what the kernels cover */
  FDLLM_ERR_CUDA = 3,          /* a CUDA runtime/driver call failed */
  FDLLM_ERR_DEVICE_BOUNDS = 4, /* a kernel found out-of-range metadata */
  FDLLM_ERR_TIMEOUT = 5        /* a bounded in-kernel wait gave up */
} fdllm_status;

typedef enum { FDLLM_BF16 = 0, FDLLM_F32 = 1 } fdllm_dtype;

/* Shape of the paged KV cache and of the layer it serves.
 *   n_layers, n_heads, head_dim, page_size, num_pages: pool geometry.
 *   hidden = n_heads * head_dim (no grouped-query attention).
 *   max_position: RoPE positions must lie in [0, max_position).
 *   rope_theta: RoPE base (rotate-half pairing (i, i + head_dim/2), angle
 *     p * rope_theta^(-2i/head_dim); [FD] paragraph 1 fuses RoPE with the
 *     projection, the form is the LLaMA-family one).
 *   max_batch, max_slots_per_seq: bounds used to size the library's
 *     attention-mass workspace (n_heads * max_batch * max_slots_per_seq
 *     floats). A step with batch > max_batch or
 *     max_blocks_per_seq * page_size > max_slots_per_seq is rejected.
 *   dtype: FDLLM_BF16 (x, Wqkv, pools in bf16; fp32 accumulation) or
 *     FDLLM_F32 (everything fp32). */
typedef struct {
  int32_t n_layers;
  int32_t n_heads;
  int32_t head_dim;
  int32_t page_size;
  int32_t num_pages;
  int32_t max_position;
  int32_t max_batch;
  int32_t max_slots_per_seq;
  float rope_theta;
  int32_t dtype; /* fdllm_dtype */
} fdllm_cache_config;

typedef struct fdllm_cache fdllm_cache; /* opaque */

/* Per-step description.
 *   batch: sequences in the step (1 .. 256).
 *   total_rows: R = cu_rows[batch].
 *   max_blocks_per_seq: row length of block_table.
 *   cu_rows: HOST int32 [batch+1], row offsets of each sequence into x/out;
 *     a sequence holds at most 128 rows.
 *   seq_lens: HOST int32 [batch], L_b = visible context slots of sequence b
 *     (slots [0, L_b) through its block table).
 *   slots: DEVICE int32 [total_rows], cache slot each row writes; NULL means
 *     slot = position.
 *   validate: 1 = copy the device metadata to the host and check it before
 *     launching (slow; for tests). Duplicate slots within a sequence and
 *     view rows writing inside [0, L_b) are only detected this way.
 *   out_bf16: 0 = `out` is fp32; 1 = `out` is bf16, each value rounded to
 *     nearest even from the kernel's fp32 result (bf16 caches only; the
 *     input of fdllm_oproj). */
typedef struct {
  int32_t batch;
  int32_t total_rows;
  int32_t max_blocks_per_seq;
  const int32_t* cu_rows;
  const int32_t* seq_lens;
  const int32_t* slots;
  int32_t validate;
  int32_t out_bf16;
} fdllm_step;

/* Creates a handle over caller-owned pools.
 *   k_pool, v_pool: DEVICE [n_layers][num_pages][n_heads][page_size][head_dim]
 *     of cfg->dtype, 16-byte aligned. Not modified here.
 * Allocates the RoPE cos/sin tables (computed on the host in double and
 * kept in double: the kernels rotate q and k in double, so each rotated
 * value is rounded to the cache dtype once), the mass workspace and a
 * device error word, and synchronises `stream` once. */
FDLLM_API fdllm_status fdllm_cache_create(const fdllm_cache_config* cfg, void* k_pool, void* v_pool,
                                void* stream, fdllm_cache** out);

/* Frees what fdllm_cache_create allocated (not the pools). NULL is a no-op. */
FDLLM_API void fdllm_cache_destroy(fdllm_cache* cache);

/* One Flash-Cache + scheduled-attention layer step ([FD] paragraphs 1-3).
 *   layer: which layer's slice of the pools to write and read.
 *   x: DEVICE [total_rows][hidden] of the cache dtype, the selected rows'
 *     hidden states (window rows, tracked rows, or the two views).
 *   wqkv: DEVICE [hidden][3*hidden] row-major; columns are [Q | K | V], each
 *     block head-major (head h at columns h*head_dim .. +head_dim-1).
 *   positions: DEVICE int32 [total_rows], RoPE positions.
 *   block_table: DEVICE int32 [batch][max_blocks_per_seq], physical page of
 *     each logical page (slot s of sequence b lives in page
 *     block_table[b][s / page_size] at offset s % page_size).
 *   view_mask: DEVICE int8 [total_rows]: 0 plain row, 1 draft view, 2 mask
 *     view; NULL = all plain. Every row sees the slots [0, L_b) as they
 *     stand after this step's writes. A view row also sees the slots that
 *     rows of its own view write in this step at positions <= its own; the
 *     two views never see each other's fresh slots. View rows must write
 *     slots >= L_b.
 *   out: DEVICE [total_rows][hidden], fp32 (or bf16 with step->out_bf16),
 *     softmax(q k^T / sqrt(head_dim)) v per head, heads concatenated.
 *   attn_mass: DEVICE fp32 [batch][max_blocks_per_seq * page_size] or NULL.
 *     attn_mass[b][s] = (1 / (R_b * n_heads)) * sum over heads and over the
 *     rows of b of the attention probability on slot s; zero for slots
 *     nobody attends. Each sequence with rows sums to 1 ([FD] paragraph 2:
 *     the statistic behind the most-attended tracking set).
 * Writes: out, attn_mass, and for every row the k/v of every head into its
 * slot; no other cache byte changes. Within one step no sequence may read a
 * slot another sequence writes.
 * A handle's device workspace (mass partials, error word) serves one step
 * at a time: steps on one handle must not run concurrently (issue them on
 * one stream, or order the streams).
 * Steps with few tiles (four CTAs per tile fit on the SMs, e.g. a single
 * sequence; hidden a multiple of 256) run each tile as a cluster of four
 * CTAs that split the projection's K range and exchange partial sums
 * through distributed shared memory; the attending CTA waits, bounded to
 * one second, for the two CTAs that write the tile's k and v rows to the
 * cache. The four CTAs of a cluster are scheduled together, so the wait
 * only runs out if that work stalls: the tile's out and attn_mass are then
 * wrong and the step records FDLLM_ERR_TIMEOUT in the device error word.
 * With step->validate = 0 the call itself still returns FDLLM_OK, so
 * callers must call fdllm_check to see it. */
FDLLM_API fdllm_status fdllm_layer_step(fdllm_cache* cache, int32_t layer, const fdllm_step* step,
                              const void* x, const void* wqkv, const int32_t* positions,
                              const int32_t* block_table, const int8_t* view_mask, void* out,
                              float* attn_mass, void* stream);

/* Next step's tracked set ([FD] paragraph 2: a fixed budget of the most
 * attended tokens).
 *   attn_mass: DEVICE fp32 [batch][row_stride], non-negative.
 *   seq_lens: DEVICE int32 [batch]; candidates are slots [0, L_b), L_b <= row_stride,
 *     L_b <= 65536.
 *   k: budget, 1 .. 1024.
 *   exclude_cu: DEVICE int32 [batch+1] or NULL; exclude_slots: DEVICE int32,
 *     slots removed from sequence b's candidates are
 *     exclude_slots[exclude_cu[b] .. exclude_cu[b+1]) (out-of-range entries
 *     are ignored).
 *   tracked: DEVICE int32 [batch][k]: the k candidates of largest mass in
 *     descending order, ties to the lower slot, padded with -1. */
FDLLM_API fdllm_status fdllm_select_tracked(const float* attn_mass, const int32_t* seq_lens, int32_t batch,
                                  int32_t row_stride, int32_t k, const int32_t* exclude_cu,
                                  const int32_t* exclude_slots, int32_t* tracked, void* stream);

/* The layer step of fdllm_layer_step without a handle and without any
 * device allocation. The paper has no counterpart: it exists for callers
 * that cannot call cudaMalloc when they run a step, such as a serving
 * engine that has already given nearly all free HBM to its KV pool, or a
 * framework whose own allocator must account for every device byte.
 *   cfg, k_pool, v_pool: as for fdllm_cache_create (same rules).
 *   rope_cos, rope_sin: DEVICE fp64 [cfg->max_position][cfg->head_dim / 2],
 *     16-byte aligned, owned by the caller: entry [p][i] is the cosine / sine
 *     of p * rope_theta^(-2i/head_dim) in double (the tables that
 *     fdllm_cache_create builds).
 *   layer, step, x, wqkv, positions, block_table, view_mask, out, attn_mass,
 *     stream: as for fdllm_layer_step; cfg->max_batch and
 *     cfg->max_slots_per_seq bound the step the same way.
 * Scratch: the per-head attention-mass partials and the device error word
 * live in one fixed 8 MiB array in the library's device image, which every
 * GPU that loads the library holds until the process exits. With attn_mass
 * non-NULL, n_heads * batch * max_blocks_per_seq * page_size must be at most
 * 2,097,088 floats, else FDLLM_ERR_UNSUPPORTED (nothing enqueued).
 * The first call on each device looks up the array's device address and
 * clears its error word, synchronising `stream` once; make that first call
 * before any stream capture. Later calls enqueue work only (no host sync
 * unless step->validate is 1).
 * Every call on a device shares the array, so calls whose work overlaps on
 * the GPU (other streams, other threads) race on it and give wrong mass or
 * error reports; serialise them. The partial rows a call uses are zeroed by
 * its own kernel, so contents left by an earlier call do not matter.
 * Errors: device-detected errors are kept in the shared error word and
 * reported, then cleared, by the next call with step->validate = 1
 * (FDLLM_ERR_DEVICE_BOUNDS or FDLLM_ERR_TIMEOUT); fdllm_check does not see
 * them. No cudaMalloc, cudaFree or other device allocation happens; host
 * planning uses ordinary host memory as in fdllm_layer_step. */
FDLLM_API fdllm_status fdllm_layer_step_noalloc(const fdllm_cache_config* cfg, void* k_pool,
                                      void* v_pool, const double* rope_cos, const double* rope_sin,
                                      int32_t layer, const fdllm_step* step, const void* x,
                                      const void* wqkv, const int32_t* positions,
                                      const int32_t* block_table, const int8_t* view_mask,
                                      void* out, float* attn_mass, void* stream);

/* Flash-Verify acceptance ([FD] paragraph 3: a block position is accepted
 * only when the draft view and the mask view agree and the mask view's
 * confidence exceeds a threshold, in causal order, stopping at the first
 * position that fails).
 *   mask_logits: DEVICE [rows][vocab] of `dtype` (FDLLM_BF16 or FDLLM_F32):
 *     the mask view's logits at the block positions; the rows of sequence b
 *     are cu_rows[b] .. cu_rows[b+1]-1, in position order. Logits must be
 *     finite or -inf, with at least one finite value per row.
 *   cu_rows: DEVICE int32 [batch+1], non-decreasing, within [0, rows].
 *   draft_tokens: DEVICE int32 [rows], the drafted token at each position.
 *   tau: confidence threshold; acceptance needs conf > tau (compared in fp32).
 *   pred: DEVICE int32 [rows] out: the most likely token (lowest id among
 *     equal largest logits).
 *   conf: DEVICE fp32 [rows] out: that token's softmax probability.
 *   n_accepted: DEVICE int32 [batch] out: the length of the accepted prefix
 *     (positions i with pred == draft and conf > tau, from the first on).
 * Reads the logits once; two launches, asynchronous on `stream`. */
FDLLM_API fdllm_status fdllm_verify_accept(const void* mask_logits, int32_t dtype, int32_t rows,
                                 int32_t vocab, const int32_t* cu_rows, int32_t batch,
                                 const int32_t* draft_tokens, float tau, int32_t* pred,
                                 float* conf, int32_t* n_accepted, void* stream);

/* Host-only: the static tile schedule the bf16 layer step uses when its
 * (row group, head) tiles outnumber the SMs. The step then launches one
 * persistent CTA per SM (per bin), which runs its bin's tiles one after
 * another; fdllm_layer_step builds this schedule itself (with the device's
 * SM count and its own per-group cost model, and caches it while the costs
 * repeat). This entry point exposes the packing for inspection and tests.
 *
 * [FD] paragraph 1 (scheduled attention over divergent lengths and stages
 * in one launch): the packing balances that launch across SMs; the pages
 * prescribe no particular packing.
 *
 *   group_cost: HOST double [n_groups], the modelled time of one tile of
 *     group g (every head's tile of a group costs the same); finite, >= 0.
 *   n_groups, n_heads: tile t = g * n_heads + h for group g, head h.
 *     At most 256 each, and n_groups * n_heads <= 1024.
 *   n_bins: number of bins (persistent CTAs), 1 .. 160.
 *   bin_start: HOST int32 [n_bins + 1] out: bin i runs
 *     tiles[bin_start[i] .. bin_start[i+1]), costliest first; bin_start[0]
 *     is 0 and bin_start[n_bins] is n_groups * n_heads.
 *   tiles: HOST int32 [n_groups * n_heads] out: every tile exactly once.
 * Packing: first-fit-decreasing into n_bins bins of the smallest capacity
 * that fits (bisection), then moves and swaps out of the fullest bin while
 * they lower it. Deterministic. Returns FDLLM_ERR_INVALID_ARG or
 * FDLLM_ERR_UNSUPPORTED outside these limits; needs no GPU. */
FDLLM_API fdllm_status fdllm_plan_tile_schedule(const double* group_cost, int32_t n_groups,
                                      int32_t n_heads, int32_t n_bins, int32_t* bin_start,
                                      int32_t* tiles);

/* Output projection of the attention block: y = residual + attn_out W_o,
 * bf16 in and out, fp32 accumulation (one tcgen05 GEMM launch).
 * [FD] paragraph 1 covers a layer up to the attention output; the
 * projection after it is the plain linear map over the heads' outputs side
 * by side, read with the conventions of wqkv (y = x W, row-major, no bias).
 * With a residual it closes the layer's attention sub-block as a
 * transformer's residual stream does (x_next = x + attn_out W_o), which is
 * how a stack of layer steps chains one layer's output into the next
 * layer's x.
 *   attn_out: DEVICE bf16 [rows][hidden], e.g. fdllm_layer_step's out with
 *     step->out_bf16 = 1. Must not overlap y.
 *   w_o: DEVICE bf16 [hidden][hidden], row-major. Must not overlap y.
 *   residual: DEVICE bf16 [rows][hidden] or NULL (no residual). It may be y
 *     itself (an in-place update of the residual stream), but may not
 *     overlap y otherwise.
 *   y: DEVICE bf16 [rows][hidden] out; each value is the fp32 sum
 *     (accumulator + residual) rounded once to nearest even.
 *   rows >= 0 (0 enqueues nothing); hidden a positive multiple of 256.
 *   All pointers 16-byte aligned.
 *   status: DEVICE int32 or NULL; a bounded in-kernel wait that gives up
 *     writes FDLLM_ERR_TIMEOUT there (and y is then incomplete); nothing
 *     else writes it.
 * Host-detectable errors return FDLLM_ERR_INVALID_ARG or
 * FDLLM_ERR_UNSUPPORTED and enqueue nothing. */
FDLLM_API fdllm_status fdllm_oproj(const void* attn_out, const void* w_o, const void* residual,
                                   void* y, int32_t rows, int32_t hidden, int32_t* status,
                                   void* stream);

/* ------------------------------------------------------------------------
 * The single-token serving step: block tables from request lengths, the
 * attention of one new token a sequence over the same paged pools, and the
 * layer's other products. [FD] covers the multi-row masked-diffusion step;
 * these are its form for a server that adds one token (or a prompt) at a
 * time to the same cache. All pointers live on the current device.
 * ------------------------------------------------------------------------ */

/* Block tables, positions and slot maps for the tokens a step adds, with
 * pages taken from a free list ([FD] paragraph 1: the block table of
 * scheduled attention). One launch, no host round trip.
 *   batch: requests (1 .. 16384). max_blocks_per_seq, page_size, num_pages:
 *     positive; (batch * max_blocks_per_seq + 1) * page_size < 2^31, and so
 *     is num_pages * page_size.
 *   capacity: room, in rows, of the four row outputs (0 .. 2^30).
 *   seq_lens: DEVICE int32 [batch], tokens each request holds.
 *   new_lens: DEVICE int32 [batch], tokens it gets now (0 allowed).
 *   block_table: DEVICE int32 [batch][max_blocks_per_seq], in and out: the
 *     entries of pages already held are read, those of new pages are
 *     written, others stay as they are.
 *   free_pages: DEVICE int32 [num_pages], the free list, of which the first
 *     n_free[0] entries are free pages; read only. Pages are taken from its
 *     end backwards, in the order of the requests, so the first
 *     n_free_out[0] entries are what remains.
 *   n_free: DEVICE int32 [1].
 * A request whose pages do not all fit (counted in request order, refused
 * ones included) is refused whole: granted 0, its length and table stay, its
 * rows have slot -1; one that needs no page is always granted.
 * Outputs (DEVICE; none may overlap an input or another output):
 *   cu_rows int32 [batch+1]: row offsets; request b's rows are
 *     cu_rows[b] .. cu_rows[b+1]-1, new_lens[b] of them (refused ones too).
 *   positions int32, slots int32, row_seq int32, slot_map int64 [capacity]:
 *     per row its position, the logical slot it writes (the position; -1 if
 *     refused), its request, and its place in the pool, page * page_size +
 *     offset (-1 if refused). positions, slots and block_table are the
 *     arguments of those names of fdllm_layer_step, which also wants host
 *     copies of cu_rows and the lengths. Entries past the last row stay as
 *     they are. The rows lie close together: a request without new tokens
 *     (or past its table's end) has none, and the entries of those behind it
 *     move up, so fdllm_decode_attention, which reads an entry a sequence,
 *     takes the outputs of fdllm_plan_step.
 *   seq_lens_out int32 [batch], granted int32 [batch], n_free_out int32 [1].
 *   headroom int32 [1] or NULL: n_free less the pages asked for by all
 *     requests up to the last granted one. It equals n_free_out unless a
 *     request before that one was refused; then it is negative, and so many
 *     pages have to come free before the refused ones among them can run.
 *     Requests refused after the last granted one do not enter it: a list
 *     that runs out and stays out shows in granted alone.
 *   status: DEVICE int32 or NULL: FDLLM_ERR_DEVICE_BOUNDS is written there
 *     for a negative length, a request past its table's end (both get no
 *     rows and granted 0), a page id outside [0, num_pages) (its rows get
 *     slot_map -1), n_free outside [0, num_pages] (clamped), or more rows
 *     than capacity (those past it are not written); nothing else writes it. */
FDLLM_API fdllm_status fdllm_plan_blocks(int32_t batch, int32_t max_blocks_per_seq,
                                         int32_t page_size, int32_t num_pages, int32_t capacity,
                                         const int32_t* seq_lens, const int32_t* new_lens,
                                         int32_t* block_table, const int32_t* free_pages,
                                         const int32_t* n_free, int32_t* cu_rows,
                                         int32_t* positions, int32_t* slots, int32_t* row_seq,
                                         int64_t* slot_map, int32_t* seq_lens_out,
                                         int32_t* granted, int32_t* n_free_out,
                                         int32_t* headroom, int32_t* status, void* stream);

/* fdllm_plan_blocks with two outputs more, an entry a request, for
 * fdllm_decode_attention over the same batch:
 *   seq_positions, seq_slots: DEVICE int32 [batch] or NULL: position and
 *     slot of the request's last row (its only one in a single-token step);
 *     0 and -1 where it has no row or was refused, so that nothing is written
 *     for it and its out means nothing.
 * A request given several tokens belongs to the multi-row step: only its
 * last one is named here. */
FDLLM_API fdllm_status fdllm_plan_step(int32_t batch, int32_t max_blocks_per_seq,
                                       int32_t page_size, int32_t num_pages, int32_t capacity,
                                       const int32_t* seq_lens, const int32_t* new_lens,
                                       int32_t* block_table, const int32_t* free_pages,
                                       const int32_t* n_free, int32_t* cu_rows,
                                       int32_t* positions, int32_t* slots, int32_t* row_seq,
                                       int64_t* slot_map, int32_t* seq_lens_out,
                                       int32_t* granted, int32_t* n_free_out,
                                       int32_t* headroom, int32_t* seq_positions,
                                       int32_t* seq_slots, int32_t* status, void* stream);

/* Gives pages back: request b keeps its first keep_lens[b] tokens (all of
 * them when that is more than it holds; 0 ends it), and the pages past them
 * go onto the free list behind its first n_free[0] entries, request by
 * request in the table's order. Used when requests finish, and when drafted
 * tokens are rejected ([FD] paragraph 3). Sizes as for fdllm_plan_blocks.
 *   block_table: DEVICE, read only; entries past the kept pages keep ids
 *     that no longer belong to the request.
 *   free_pages: DEVICE int32 [num_pages], in and out.
 *   seq_lens_out, n_free_out: DEVICE, out; must not overlap an input.
 *   status: FDLLM_ERR_DEVICE_BOUNDS for a negative length, a length past the
 *     table's end (such a request gives nothing back), a page id outside
 *     [0, num_pages) (listed as -1) or a list that would grow past num_pages
 *     (the pages past it are dropped). */
FDLLM_API fdllm_status fdllm_release_blocks(int32_t batch, int32_t max_blocks_per_seq,
                                            int32_t page_size, int32_t num_pages,
                                            const int32_t* seq_lens, const int32_t* keep_lens,
                                            const int32_t* block_table, int32_t* free_pages,
                                            const int32_t* n_free, int32_t* seq_lens_out,
                                            int32_t* n_free_out, int32_t* status, void* stream);

/* Shape of a decode-attention call.
 *   batch: sequences, one query token each (>= 1).
 *   n_heads: query heads, a multiple of n_kv_heads (query head h reads key
 *     head h / (n_heads / n_kv_heads)).
 *   head_dim: 32, 64, 96 or 128.
 *   n_layers, num_pages, page_size, n_kv_heads: pool geometry, as in
 *     fdllm_cache_config with n_kv_heads for n_heads; any page size. The
 *     table's slots in tiles of 64 (bf16) or 32 (fp32), times batch and
 *     key heads (once for every 8 query heads of one), stay below 2^31.
 *   max_position: rows of the RoPE tables (ignored without them).
 *   dtype: of the pools (fdllm_dtype). in_dtype: of q, k and v.
 *   out_dtype: of out.
 *   scale: factor of the scores, finite and > 0.
 *   q_stride, k_stride, v_stride: elements between the sequences' rows. */
typedef struct {
  int32_t batch;
  int32_t n_heads;
  int32_t n_kv_heads;
  int32_t head_dim;
  int32_t n_layers;
  int32_t num_pages;
  int32_t page_size;
  int32_t max_blocks_per_seq;
  int32_t max_position;
  int32_t dtype;
  int32_t in_dtype;
  int32_t out_dtype;
  float scale;
  int64_t q_stride;
  int64_t k_stride;
  int64_t v_stride;
} fdllm_decode;

/* Device workspace, in bytes, that fdllm_decode_attention needs for these
 * heads on the current device, whatever the batch and the lengths; -1 for a
 * shape it does not serve. */
FDLLM_API int64_t fdllm_decode_workspace_bytes(int32_t n_heads, int32_t n_kv_heads,
                                               int32_t head_dim);

/* Attention of one new token a sequence over its pages: RoPE of q and k, the
 * cache write of k and v, then out = softmax(scale q' k^T) v over the slots
 * [starts[b], seq_lens[b]) as they stand after the write ([FD] paragraph 1
 * for a single row a sequence; the work is split over the slots).
 *   q: DEVICE [batch][n_heads * head_dim] of in_dtype, rows q_stride apart.
 *   k, v: DEVICE [batch][n_kv_heads * head_dim] of in_dtype, rows k_stride /
 *     v_stride apart, or both NULL: nothing is written to the cache.
 *     q, k, v may be slices of one buffer; pointers and row strides (in
 *     bytes) are multiples of 16.
 *   positions: DEVICE int32 [batch]; needed with the RoPE tables, and with k
 *     when slots is NULL (seq_positions of fdllm_plan_step).
 *   slots: DEVICE int32 [batch], the slot the new k and v go to (seq_slots of
 *     fdllm_plan_step), or NULL: slot = position. A negative slot writes nothing. No two sequences may
 *     write one place of the pool, and none may see a slot that another
 *     sequence writes in this call.
 *   rope_cos, rope_sin: DEVICE fp64 [max_position][head_dim / 2], as for
 *     fdllm_layer_step_noalloc, 16-byte aligned; both NULL: q and k are
 *     taken as they are. k is rounded to the pool's dtype once; q is not.
 *   k_pool, v_pool: DEVICE pools as for fdllm_cache_create, 16-byte aligned;
 *     at most the rows (k, v) change.
 *   block_table: DEVICE int32 [batch][max_blocks_per_seq].
 *   seq_lens: DEVICE int32 [batch], visible slots, the new token's included
 *     when it is to see itself. 0: nothing is visible.
 *   starts: DEVICE int32 [batch], first visible slot, or NULL: 0.
 *   out: DEVICE [batch][n_heads * head_dim] of out_dtype; zeros for a
 *     sequence that sees nothing. lse: DEVICE fp32 [batch][n_heads] or NULL:
 *     the natural log of the sum of exp(scores); -inf where nothing is seen.
 *   workspace: DEVICE, workspace_bytes >= fdllm_decode_workspace_bytes,
 *     16-byte aligned; no initial contents needed. Calls that may run at the
 *     same time need workspaces of their own.
 *   status: DEVICE int32 or NULL: FDLLM_ERR_DEVICE_BOUNDS is written there
 *     for a length outside [0, max_blocks_per_seq * page_size], a position
 *     outside the tables or a slot past the block table (such a sequence
 *     writes nothing and its out is zero), and for a page id outside
 *     [0, num_pages) (its slots are left out); FDLLM_ERR_TIMEOUT when a
 *     bounded in-kernel wait gives up (out and lse are then incomplete).
 *     Nothing else writes it. Without it such errors are not reported.
 * Sums and softmax statistics are fp32. With a bf16 pool q' and the
 * probabilities enter the products as pairs of bf16 (16 bits). Results do
 * not depend on the order in which the GPU runs the CTAs. A NaN score makes
 * that head's out and lse NaN; so may an infinite k or v in a visible slot,
 * whose product with the low half of a pair is one. Two launches. */
FDLLM_API fdllm_status fdllm_decode_attention(
    const fdllm_decode* shape, int32_t layer, const void* q, const void* k, const void* v,
    const int32_t* positions, const int32_t* slots, const double* rope_cos,
    const double* rope_sin, void* k_pool, void* v_pool, const int32_t* block_table,
    const int32_t* seq_lens, const int32_t* starts, void* out, float* lse, void* workspace,
    int64_t workspace_bytes, int32_t* status, void* stream);

/* Activations: relu(a); silu(a) = a / (1 + e^-a); gelu(a) = a/2 (1 +
 * erf(a / sqrt 2)); gelu_tanh(a) = a/2 (1 + tanh(sqrt(2/pi) (a + 0.044715
 * a^3))). In fp32: silu to 2^-19 of its value; the gelus as written, to about
 * 2^-22 of |a|, which for a below -3 or so is more than that of the value. */
typedef enum {
  FDLLM_ACT_NONE = 0,
  FDLLM_ACT_RELU = 1,
  FDLLM_ACT_SILU = 2,
  FDLLM_ACT_GELU = 3,
  FDLLM_ACT_GELU_TANH = 4
} fdllm_act;

/* Shape of a linear call.
 *   rows >= 0 (0 enqueues nothing), at most 2^23. n_in, n_out: positive
 *     multiples of 8, at most 2^20.
 *   act: fdllm_act. bias_dtype: of bias and bias_gate. out_dtype: of y.
 *   ldx, ldr, ldy: elements between the rows of x, residual and y, at least
 *     n_in, n_out and n_out; rows start on 16-byte boundaries. */
typedef struct {
  int32_t rows;
  int32_t n_in;
  int32_t n_out;
  int32_t act;
  int32_t bias_dtype;
  int32_t out_dtype;
  int64_t ldx;
  int64_t ldr;
  int64_t ldy;
} fdllm_linear_shape;

/* y = residual + act(x w + bias), or with w_gate
 * y = residual + act(x w_gate + bias_gate) * (x w + bias): a layer's
 * projections and the first half of its (gated) feed-forward block, in one
 * launch. fdllm_oproj is its special case of a square w. This call is the
 * faster one but for 1000 to 1500 rows of small squares (4096 x 4096: 9.7 us
 * against 24 for one row, 18 against 26 for 256, 99 against 127 for 4096;
 * 1024 x 1024: 4.4 against 8.4 for one row, 11.5 against 10.4 for 1536).
 *   x: DEVICE bf16 [rows][n_in]. w, w_gate: DEVICE bf16 [n_in][n_out],
 *     row-major and contiguous (y = x W, as wqkv); w_gate may be NULL.
 *   bias, bias_gate: DEVICE [n_out] of bias_dtype, or NULL; bias_gate needs
 *     w_gate.
 *   residual: DEVICE bf16 [rows][n_out] or NULL. It may be y itself (same
 *     pointer, stride and type), but may not overlap y otherwise.
 *   y: DEVICE [rows][n_out] of out_dtype; overlaps no other argument (an
 *     argument reaches from its first to its last element, the gaps between
 *     its rows included).
 *   All pointers 16-byte aligned (biases too).
 *   status: DEVICE int32 or NULL; a bounded in-kernel wait that gives up
 *     writes FDLLM_ERR_TIMEOUT there (y is then incomplete).
 * Sums, bias, activation, product and residual are fp32; y is rounded once. */
FDLLM_API fdllm_status fdllm_linear(const fdllm_linear_shape* shape, const void* x, const void* w,
                                    const void* bias, const void* w_gate, const void* bias_gate,
                                    const void* residual, void* y, int32_t* status, void* stream);

/* Synchronises `stream`, reads and clears the handle's device error word.
 * Returns FDLLM_OK, FDLLM_ERR_DEVICE_BOUNDS, FDLLM_ERR_TIMEOUT or
 * FDLLM_ERR_CUDA. */
FDLLM_API fdllm_status fdllm_check(fdllm_cache* cache, void* stream);

/* Failure injection for tests of the error path (the paper has no
 * counterpart). Faults are made on the host; nothing here traps, faults or
 * hangs the GPU.
 *   FDLLM_INJECT_SPLIT_FLAG_TIMEOUT: in the next fdllm_layer_step on `cache`
 *     that runs its tiles as four-CTA clusters, the k / v writing CTAs
 *     withhold their signal to the attending CTA, whose wait is bounded to
 *     `wait_ns` nanoseconds (1 .. 1e9) instead of one second. When it runs out
 *     the CTA records FDLLM_ERR_TIMEOUT in the device error word and skips
 *     its attention, issuing no further load or product; that step's out
 *     rows are left unwritten and its attention mass is zero. The next
 *     fdllm_check returns FDLLM_ERR_TIMEOUT and clears the word; the handle
 *     stays usable. The injection applies once, and stays pending while
 *     steps do not split their tiles.
 *   FDLLM_INJECT_NONE: cancels a pending injection.
 * Returns FDLLM_ERR_INVALID_ARG for a null handle, an unknown kind or a
 * wait outside the range. */
typedef enum { FDLLM_INJECT_NONE = 0, FDLLM_INJECT_SPLIT_FLAG_TIMEOUT = 1 } fdllm_inject_kind;
FDLLM_API fdllm_status fdllm_inject_fault(fdllm_cache* cache, int32_t kind, int64_t wait_ns);

/* The same for the single-token calls, which have no handle: the next
 * fdllm_decode_attention or fdllm_linear of this thread that enqueues work
 * says of the first tile of every CTA that it is not there (its copies are
 * made and waited for), and bounds its waits to about wait_ns nanoseconds
 * (1 .. 1e9) instead of a second. They run out, FDLLM_ERR_TIMEOUT is written to
 * that call's status, and its output is incomplete (k and v may not be in the
 * cache). Applies once; 0 cancels it. */
FDLLM_API fdllm_status fdllm_inject_tile_timeout(int64_t wait_ns);

/* Static description of a status code. */
FDLLM_API const char* fdllm_status_string(fdllm_status status);

/* Message for the last failing call on this thread ("" if none). */
FDLLM_API const char* fdllm_last_error(void);

/* Number of kernel launches the last successful fdllm_layer_step,
 * fdllm_layer_step_noalloc, fdllm_select_tracked, fdllm_verify_accept,
 * fdllm_oproj, fdllm_plan_blocks, fdllm_plan_step, fdllm_release_blocks,
 * fdllm_decode_attention or fdllm_linear call on this thread enqueued. */
FDLLM_API int32_t fdllm_last_launch_count(void);

#ifdef __cplusplus
}
#endif

#endif /* FDLLM_H */
