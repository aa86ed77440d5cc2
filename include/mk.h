/*
 * mk.h -- C ABI of the GB300 (sm_103a) MoE token dispatch + expert GEMM.
 *
 * What the operation is.  The mKernel write-ups name "MoE Dispatch+GEMM" as
 * one of five fused persistent kernels: tokens are routed dynamically to
 * experts and each expert's dense product runs as soon as its tile of tokens
 * has arrived, inside one kernel ("mKernel: UCCL fuses NVLink, RDMA and
 * compute into one persistent CUDA kernel", zubnet.ai, paras. 1-2;
 * "UC Berkeley presenta mKernel ...", edge.aivizor.me, para. 3;
 * "mKernel : une bibliotheque de noyaux fusionnes ...", lefilia.fr,
 * paras. 1 and 3).  The pages print none of the steps, so this header
 * states the contract the library implements:
 *
 *   1. Router top-k.  For token t, the k experts with the largest logits,
 *      in descending order, ties to the lower expert id; -inf is a legal
 *      logit (NaN and +inf are outside the contract: results unspecified,
 *      no fault).
 *   2. Gates.  gate[t,j] = softmax over the k chosen logits (fp32 expf);
 *      a -inf logit gets 0; if all k chosen are -inf every gate is 0.
 *   3. expert_offsets[e] = number of (t,j) routed to experts < e
 *      (exclusive scan of the per-expert histogram); expert_offsets[E] = T*k.
 *   4. Sorted rows: every (t,j) pair, ordered by (expert, t, j).  For sorted
 *      row r: src_index[r] = t*k + j, gate_w[r] = gate[t,j].
 *   5. y_sorted[r,:] = x[t,:] . W[e,:,:] with fp32 accumulation, stored as
 *      bf16 (round-to-nearest-even) or, with MK_OUT_F32, as fp32.  Rows are
 *      not scaled by the gate.
 *
 * Layouts (all row-major, caller-owned, device memory unless stated):
 *   x[T,H] bf16, logits[T,E] f32, W[E,H,F] bf16 (F contiguous)   -- read only
 *   y_sorted[T*k,F] bf16 (or f32), src_index[T*k] i32,
 *   expert_offsets[E+1] i32, gate_w[T*k] f32                     -- written
 *   bf16 travels as 16-bit storage (void*); the library never frees caller
 *   memory.
 *
 * Limits (checked synchronously, no launch on failure -> MK_ERR_INVALID_ARG
 * or MK_ERR_UNSUPPORTED): T >= 0; 1 <= k <= min(E, 8); 1 <= E <= 256;
 * H and F multiples of 64 in [64, 32768]; T*k < 2^31; x, W, y_sorted 16-byte
 * aligned, the other arrays 4-byte aligned; the current device must be
 * sm_103 (compute capability 10.3).  T == 0 is valid: expert_offsets is set
 * to zeros and nothing else is written.
 *
 * Asynchrony.  Calls enqueue work on `stream` (a cudaStream_t; NULL is the
 * legacy default stream) and return without synchronising.  A fault or a
 * bounded wait that ran out inside the kernel is recorded in a per-device
 * error word; mk_get_status() synchronises the stream and reports it.
 *
 * Threads.  Calls may come from several host threads; those that use the
 * library's workspace of one stream are enqueued one after another.  The
 * per-thread default stream has a workspace in each thread that used it, kept
 * until mk_release_workspace().  A call on a new stream that got the handle of
 * a destroyed one waits for the device once.
 */
#ifndef MK_H
#define MK_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MK_OK = 0,
    MK_ERR_INVALID_ARG = 1,   /* bad size, null or misaligned pointer      */
    MK_ERR_UNSUPPORTED = 2,   /* wrong device, or shape beyond the limits  */
    MK_ERR_CUDA = 3,          /* a CUDA runtime call failed                */
    MK_ERR_TIMEOUT = 4,       /* a bounded device wait ran out             */
    MK_ERR_DEVICE_FAULT = 5,  /* the kernel detected an inconsistent state */
    MK_ERR_NOT_IMPLEMENTED = 6,
    MK_ERR_WORKSPACE = 7      /* caller workspace too small or misaligned  */
} mk_status_t;

/* Execution modes. */
enum {
    MK_MODE_FUSED = 0,         /* one persistent launch: dispatch and compute roles overlap per tile */
    MK_MODE_UNFUSED = 1,       /* the same steps as four launches (route, scan, gather, GEMM)       */
    MK_MODE_DISPATCH_ONLY = 2  /* routing + gather only (y_sorted untouched); measures dispatch      */
};

enum { MK_OUT_BF16 = 0, MK_OUT_F32 = 1 };

/* Host-side fault injection (never a device trap): withhold the arrival of
 * one tile's rows (its readiness never completes) so the compute role's
 * bounded wait runs out.  It acts on staged rows: with the fault set, AUTO
 * row sources resolve to MK_GATHER_STAGED. */
enum { MK_FAULT_NONE = 0, MK_FAULT_DROP_TILE_FLAG = 1 };

typedef struct mk_config {
    int32_t mode;           /* MK_MODE_*                                        */
    int32_t out_dtype;      /* MK_OUT_BF16 or MK_OUT_F32                         */
    int32_t dispatch_ctas;  /* CTAs in the dispatch role; 0 = shape heuristic    */
    int32_t grid_ctas;      /* persistent grid size; 0 = one CTA per SM          */
    int32_t n_group;        /* N-blocks per group in the work order; 0 = auto    */
    int32_t debug_fault;    /* MK_FAULT_*                                        */
    int64_t spin_limit_ns;  /* bound on every device wait; 0 = 2 s               */
    int32_t trace;          /* 1 = record per-CTA %globaltimer phase stamps      */
    int32_t l2_prefetch;    /* W K-blocks prefetched into L2 ahead of use;
                               <= 0 = off (the default)                          */
    int32_t mma_pair;       /* MK_MMA_*: one SM per 128-row tile, an SM pair
                               (cta_group::2) per 256-row tile, or one SM per
                               256-row tile with two accumulators (WIDE)     */
    int32_t gather;         /* MK_GATHER_*: where the GEMM's token rows come from */
    int32_t reserved[4];    /* must be zero                                     */
} mk_config_t;

/* Token rows for the GEMM.  STAGED: dispatch CTAs copy them into
 * expert-contiguous tiles in the workspace, in units of up to 32 rows, and
 * add each unit's rows to its tile's arrival count; compute CTAs wait until
 * a tile's count reaches its rows and load whole tiles.  DIRECT: the GEMM's
 * producer warp copies each tile's rows straight from x into its
 * shared-memory stages (16-byte cp.async), so there is no staging copy, no
 * gather role, and the workspace holds no staging rows (T*k*H*2 bytes
 * less); 128-row or wide tiles (not SM pairs), and T*H*2 < 4 GiB.  GATHER4:
 * as DIRECT, but the rows arrive by TMA tile::gather4 (four token rows per
 * instruction, one instruction per lane of the producer warp) instead of
 * cp.async; same tiles and limits.  AUTO: DIRECT when k >= 4 and
 * T*k >= 256*E (wide tiles), or when the staged rows would take under
 * 1 MiB (T*k*H*2 < 2^20), with cfg.mma_pair AUTO or WIDE and
 * T*H*2 < 4 GiB; STAGED otherwise.  The expert-parallel entry points stage
 * rows (DIRECT and GATHER4 return MK_ERR_UNSUPPORTED there). */
enum { MK_GATHER_AUTO = 0, MK_GATHER_STAGED = 1, MK_GATHER_DIRECT = 2, MK_GATHER_GATHER4 = 3 };

/* Expert GEMM tile.  SINGLE: each CTA runs a 128 x 256 tile alone.  PAIR: a
 * cluster of two CTAs (two SMs) runs a 256 x 256 tile with the 2-SM tensor
 * core instruction; each SM stages half the operands, so the same shared
 * memory holds six stages instead of four.  WIDE: each CTA runs a 256 x 256
 * tile alone, as two 128-row accumulators that share every staged block of
 * the weights (three stages of 64 KiB; an expert's last tile of at most 128
 * rows uses one accumulator); with any MK_GATHER_* form.  AUTO: WIDE when
 * T*k >= 256*E (two or more 128-row tiles per expert on average), SINGLE
 * otherwise. */
enum { MK_MMA_AUTO = 0, MK_MMA_SINGLE = 1, MK_MMA_PAIR = 2, MK_MMA_WIDE = 3 };

/* Per-launch facts, for tests and the benchmark. */
typedef struct mk_launch_info {
    int32_t grid_ctas;      /* CTAs launched by the persistent kernel */
    int32_t dispatch_ctas;  /* of which in the dispatch role          */
    int32_t launches;       /* kernels launched by the last call      */
    int32_t n_group;
    int64_t workspace_bytes;
    int32_t mma_pair;       /* MK_MMA_SINGLE, MK_MMA_PAIR or MK_MMA_WIDE as resolved */
    int32_t gather;         /* MK_GATHER_STAGED, _DIRECT or _GATHER4 as resolved */
    int32_t route_lanes;    /* lanes sharing each token's experts in routing (1, 2, 4, 8) */
    int32_t route_chunks;   /* routing chunks (224 / route_lanes tokens each) */
} mk_launch_info_t;

/* Fill `cfg` with the defaults (fused, bf16 output, heuristic split). */
void mk_config_default(mk_config_t* cfg);

/* The fused path with default configuration and the library's
 * per-(device, stream) workspace cache.  Device pointers; see above. */
mk_status_t mk_moe_dispatch_gemm(const void* x, const float* logits, int T, int H, int E, int k,
                                 const void* W, int F, void* y_sorted, int32_t* src_index,
                                 int32_t* expert_offsets, float* gate_w, void* stream);

/* As mk_moe_dispatch_gemm with an explicit configuration (NULL = defaults)
 * and an optional caller workspace.  With workspace == NULL the library's
 * cache is used (grown with cudaMallocAsync on `stream`; under stream capture
 * a buffer of the cache that is large enough becomes the captured calls', else
 * the graph allocates and frees its own).  A caller
 * workspace must hold mk_workspace_size() bytes, be 256-byte aligned, and be
 * zero-filled before its first use (the kernels leave it ready for the next
 * call).  One workspace serves one stream at a time. */
mk_status_t mk_moe_dispatch_gemm_ex(const void* x, const float* logits, int T, int H, int E, int k,
                                    const void* W, int F, void* y_sorted, int32_t* src_index,
                                    int32_t* expert_offsets, float* gate_w, void* stream,
                                    const mk_config_t* cfg, void* workspace, size_t ws_bytes);

/* The path plus the combine that completes an MoE layer: after the expert
 * products, out[t,:] = sum_j gate[t,j] * y_sorted[row of (t,j), :] (fp32,
 * slots in order, no atomics), in y_sorted's dtype (bf16, or f32 with
 * MK_OUT_F32).  The pages name the operation "MoE Dispatch+GEMM" and route
 * each token to experts ("mKernel : une bibliotheque ...", lefilia.fr,
 * para. 3); this weighted sum of a token's expert outputs is the textbook
 * step that follows.  out[T,F]: device, caller-owned, 16-byte aligned.
 * Fused mode combines inside the same persistent launch after a grid
 * barrier; unfused mode adds a fifth launch.  y_sorted and the other outputs
 * are written as by mk_moe_dispatch_gemm_ex.  Not valid with
 * MK_MODE_DISPATCH_ONLY. */
mk_status_t mk_moe_dispatch_gemm_combine(const void* x, const float* logits, int T, int H, int E, int k,
                                         const void* W, int F, void* y_sorted, int32_t* src_index,
                                         int32_t* expert_offsets, float* gate_w, void* out, void* stream,
                                         const mk_config_t* cfg, void* workspace, size_t ws_bytes);

/* Gated expert FFN (SwiGLU, the Mixtral / DeepSeek expert shape; both model
 * families are named in "mKernel : une bibliotheque de noyaux fusionnes
 * ...", lefilia.fr, para. 3): the same dispatch, then for sorted row r of
 * token t routed to expert e,
 *   h_sorted[r,:] = silu(x[t,:] . W1[e]) * (x[t,:] . W3[e]),  silu(a) = a / (1 + e^-a),
 * both products accumulated in fp32 in the same tensor-core pass (the A tile
 * is shared; 128 columns of each projection per work item) and the SwiGLU
 * applied in the epilogue (fp32, fast exponential and divide) before
 * rounding to bf16 (or f32 with MK_OUT_F32).  W1, W3: [E,H,F] bf16, device,
 * 16-byte aligned.  Runs on tiles of one SM, 128-row or wide (MK_MMA_PAIR
 * returns MK_ERR_UNSUPPORTED).  Other
 * arguments and outputs as for mk_moe_dispatch_gemm_ex. */
mk_status_t mk_moe_dispatch_gated(const void* x, const float* logits, int T, int H, int E, int k, const void* W1,
                                  const void* W3, int F, void* h_sorted, int32_t* src_index,
                                  int32_t* expert_offsets, float* gate_w, void* stream, const mk_config_t* cfg,
                                  void* workspace, size_t ws_bytes);

/* Expert parallelism simulated on one GPU.  The pages run MoE
 * Dispatch+GEMM across GPUs, tokens travelling to the GPU that holds their
 * expert ("mKernel: UCCL fuses NVLink, RDMA, compute ...", zubnet.ai, para.
 * 2; "mKernel : une bibliotheque ...", lefilia.fr, paras. 2-3).  Here
 * `ranks` logical ranks share one launch, each with its own region of the
 * workspace standing for its device memory.  Rank r owns the tokens
 * [floor(r*T/R), floor((r+1)*T/R)) and the experts [r*E/R, (r+1)*E/R)
 * (R = ranks, 1..8, dividing E).  Each rank routes its own tokens, sends
 * its per-expert count rows to every rank (a flag per source), sends each
 * routed row to the rank of its expert (a count of arrived rows per tile:
 * the GEMM starts a tile once every source's rows are in), runs the expert
 * GEMM for its own experts, and stores every result back into the sending
 * rank's rows; with `out`, each rank then combines its own tokens once all
 * their results are back.
 *
 * Outputs (device, caller-owned, written):
 *   y_tok[T*k,F]: the product x[t].W[e] of entry (t, j) at row t*k + j
 *     (token-major: the sending ranks' return rows, rank r's being rows
 *     [T0(r)*k, T0(r+1)*k)); bf16, or f32 with MK_OUT_F32.  Not gate-scaled.
 *   src_index[T*k], gate_w[T*k], expert_offsets[E+1]: the ranks' receive
 *     buffers one after another, which is exactly the sorted order of
 *     mk_moe_dispatch_gemm (rank q's rows are [expert_offsets[q*E/R],
 *     expert_offsets[(q+1)*E/R])).
 *   out[T,F] (optional, may be NULL): sum_j gate[t,j] * y_tok[t*k+j], fp32
 *     in slot order, in y_tok's dtype.
 * Supported: MK_MODE_FUSED, staged rows, tiles of one SM (128-row or
 * wide, resolved as for the single-device call); other choices
 * return MK_ERR_UNSUPPORTED.  cfg.trace records nothing here.  workspace:
 * NULL (library cache, zeroed when allocated) or mk_ep_workspace_size()
 * bytes, 256-byte aligned, zero-filled before its first use, and used by
 * this entry point only (the others write over its control blocks).  Every rank may
 * receive up to T*min(k, E/R) rows, so the workspace holds that many
 * H-wide rows per rank.  Errors as for mk_moe_dispatch_gemm_ex. */
mk_status_t mk_moe_ep_sim(const void* x, const float* logits, int T, int H, int E, int k, const void* W, int F,
                          int ranks, void* y_tok, int32_t* src_index, int32_t* expert_offsets, float* gate_w,
                          void* out, void* stream, const mk_config_t* cfg, void* workspace, size_t ws_bytes);

/* The gated (SwiGLU) expert FFN of mk_moe_dispatch_gated under the same
 * expert-parallel simulation: each rank computes
 * h = silu(x[t].W1[e]) * (x[t].W3[e]) for the rows it received and returns
 * them to the sending ranks (h_tok[t*k + j]); with `out`, each rank combines
 * its own tokens' h rows.  W1, W3: [E,H,F] bf16, device, 16-byte aligned.
 * Other arguments, outputs and errors as for mk_moe_ep_sim; the workspace
 * is the same size. */
mk_status_t mk_moe_ep_sim_gated(const void* x, const float* logits, int T, int H, int E, int k, const void* W1,
                                const void* W3, int F, int ranks, void* h_tok, int32_t* src_index,
                                int32_t* expert_offsets, float* gate_w, void* out, void* stream,
                                const mk_config_t* cfg, void* workspace, size_t ws_bytes);

/* Workspace bytes mk_moe_ep_sim needs (0 for invalid sizes). */
size_t mk_ep_workspace_size(int T, int H, int F, int E, int k, int ranks);

/* End-to-end variant: x, logits and the four outputs are HOST buffers
 * (pinned memory gives asynchronous copies); W stays on the device (expert
 * weights are resident).  Copies the inputs in, runs the fused path, copies
 * the outputs back, and synchronises `stream` before returning, so the host
 * buffers are ready on return.  With the fused single-SM path, y_sorted goes
 * back in chunks of sorted rows (whole 256-row tiles, at most 64 chunks)
 * while the kernel still runs: the kernel raises a flag per finished chunk
 * and a second, library-owned stream waits on the flags and copies the rows,
 * in copies of 1, 1, 2, 4, ... chunks; other configurations copy after the
 * kernel.  With cfg->n_group = 0 this call orders the work tile by tile
 * (all N-blocks of a tile together), so rows complete in order.  Device
 * staging comes from the library cache.  It, the library's stream and the
 * chunk flags belong to (device, stream); calls on one stream run one after
 * another, from whichever host threads they come. */
mk_status_t mk_moe_dispatch_gemm_host(const void* x_host, const float* logits_host, int T, int H, int E,
                                      int k, const void* W, int F, void* y_sorted_host,
                                      int32_t* src_index_host, int32_t* expert_offsets_host,
                                      float* gate_w_host, void* stream, const mk_config_t* cfg);

/* Size of the fixed device array that mk_moe_dispatch_gemm_noalloc works in. */
#define MK_NOALLOC_SCRATCH_BYTES (64u << 20)

/* Allocation-free variant of mk_moe_dispatch_gemm_ex (the pages have no
 * counterpart: it serves callers of this library that may not allocate
 * device memory while they run it -- a host framework that owns the whole
 * device-memory budget through its own allocator, or a latency-critical
 * decode loop where cudaMalloc and its possible device-wide synchronisation
 * are not allowed).  Same arguments and outputs as the allocating path; the
 * caller still passes every input and output.  Instead of a workspace it
 * uses one static device array of MK_NOALLOC_SCRATCH_BYTES (64 MiB), which
 * each GPU where it is set up keeps until the process exits.  Calls whose
 * mk_workspace_size() exceeds that return MK_ERR_WORKSPACE and launch
 * nothing (it fits decode-sized batches: about T*k*H*2 bytes of staged rows
 * plus small tables).  No cudaMalloc, cudaFree or allocating library call
 * is made.  The first call on a device looks up the array's device address
 * (cudaGetSymbolAddress, with that device current) and keeps it; make that
 * first call before any stream capture.  After a device reset
 * (cudaDeviceReset), call mk_release_workspace() before the next call: it
 * drops the kept addresses (the array may sit elsewhere in the new context)
 * as well as the workspace cache.  Every call on a device shares the array
 * and finds the previous call's contents there (the call clears what must
 * start at zero), so calls that overlap on the GPU -- on different streams,
 * or from different threads -- race: serialise them.  cfg->trace must be 0
 * (MK_ERR_UNSUPPORTED otherwise): phase stamps would land in the array,
 * where mk_read_trace cannot reach them. */
mk_status_t mk_moe_dispatch_gemm_noalloc(const void* x, const float* logits, int T, int H, int E, int k,
                                         const void* W, int F, void* y_sorted, int32_t* src_index,
                                         int32_t* expert_offsets, float* gate_w, void* stream,
                                         const mk_config_t* cfg);

/* Bytes of workspace a call with these sizes needs (0 on invalid sizes). */
size_t mk_workspace_size(int T, int H, int F, int E, int k, const mk_config_t* cfg);

/* ------------------------------------------------------------------------
 * Operators of a decode step around the expert layer.  All of them: device
 * pointers, caller-owned; work is enqueued on `stream` and the call returns
 * without synchronising; arguments are checked first and nothing is launched
 * on a failure (MK_ERR_INVALID_ARG, MK_ERR_UNSUPPORTED); a device of compute
 * capability 10.3.  Sums, norms and softmax statistics are held in fp32 and
 * each output is rounded once from them; the operands of products that have
 * fewer bits (h, the attention's weights) are named at their entry.  Equal
 * inputs give equal bits.
 *
 * They can be captured in a CUDA graph.  Under capture the library's
 * workspace cache is not grown (MK_ERR_WORKSPACE): make a call of the same
 * sizes on that stream before, and order replays after it.  The buffer that a
 * captured call uses belongs from then on to the captured calls of its stream
 * (later calls get another) and stays until mk_release_workspace(): replay no
 * two graphs of one stream at a time, or capture with a caller workspace. */

/* The residual's addition and the root-mean-square norm, in bf16 and / or in
 * 8 bits.  With z = x + residual (x alone when residual is NULL):
 *   residual_out[t,:] = bf16(z),
 *   y = z * rsqrt(mean(z^2) + eps) * weight,
 *   out[t,:] = bf16(y),
 *   for each group of 128 columns (the last may be shorter): a = max |y|,
 *   scale[t,g] = a / 448 (1 when a < 2^-100), out8[t,:] = e4m3(y / scale).
 * y comes from the unrounded z.  A NaN in a row makes the row's y and scales
 * NaN.
 *   x[T,H] bf16 with x_stride elements between rows, residual[T,H] bf16 with
 *   residual_stride (may be NULL), weight[H] bf16                 -- read only
 *   out[T,H] bf16, out8[T,H] e4m3 with scale[T, ceil(H/128)] f32 (either of
 *   the two outputs may be NULL; out8 and scale come together),
 *   residual_out[T,H] bf16 (may be NULL; needs residual)          -- written
 * residual_out may be residual itself when residual_stride is H; other
 * overlaps of inputs and outputs are not allowed.  1 <= H <= 32768 (odd
 * widths too), T >= 0, eps >= 0 and finite, strides of at least H when
 * T > 1.  Rows that are 16-byte aligned (H, strides and pointers) are read
 * 16 bytes at a time. */
mk_status_t mk_add_rmsnorm(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                           const void* weight, int T, int H, float eps, void* out, void* out8, float* scale,
                           void* residual_out, void* stream);

/* Attention of one new token per sequence over a paged key-value cache.  For
 * sequence b with n = seq_lens[b] cached keys (the new token's own among
 * them), query head h and its key-value head c = h / (Hq/Hkv):
 *   s_j = scale * q[b,h,:] . k(j,c,:)  for j < n,   m = max_j s_j,
 *   out[b,h,:] = sum_j e^(s_j - m) v(j,c,:) / sum_j e^(s_j - m),
 *   lse[b,h] = log sum_j e^(s_j);
 * without keys (n = 0, or every score -inf) out is 0 and lse -inf.  The weight
 * e^(s_j - m) enters the product with v with 16 significant bits, its sum with
 * 24 (the exponential is off by 2^-21 of it at most).  Key j of
 * sequence b lies in page block_table[b, j / page_size] at token
 * j % page_size: element page*page_stride + token*token_stride +
 * c*head_stride of k_cache and of v_cache, D elements in a row.  Nothing past
 * the n-th key is read, whatever the pages hold there.
 *   q[B,Hq,D] bf16 with q_stride elements between sequences (heads
 *   contiguous), caches bf16, block_table[B,max_pages] i32 (entries past a
 *   sequence's pages are not read), seq_lens[B] i32 (device)      -- read only
 *   out[B,Hq,D] bf16, lse[B,Hq] f32 (may be NULL)                 -- written
 * Limits: D = 64, 128 or 256; Hq a multiple of Hkv; any page_size >= 1;
 * B <= 4096; max_pages*page_size <= 2^31 - 32, and fewer than 2^31 tiles of
 * 16 keys and 16 query heads in all; strides non-negative multiples of 8
 * elements, caches 16-byte aligned, out 8, q 4 (q_stride even).  Infinite
 * values give infinite outputs (one whose weight is below 2^-100 of the
 * largest may give NaN); a score that is NaN or +inf makes its head's out and
 * lse NaN.  The lengths and pages are checked on the
 * device: a length outside [0, max_pages*page_size] is clamped, a page
 * outside [0, num_pages) is not read (its keys count as zeros), and either is
 * reported by mk_get_status() as MK_ERR_DEVICE_FAULT.
 * workspace: NULL (library cache) or mk_paged_attention_workspace_size()
 * bytes, 256-byte aligned, zero-filled before its first use and used by this
 * entry point only; one stream at a time. */
mk_status_t mk_paged_attention(const void* q, int64_t q_stride, const void* k_cache, const void* v_cache,
                               int64_t page_stride, int64_t token_stride, int64_t head_stride,
                               const int32_t* block_table, const int32_t* seq_lens, int B, int Hq, int Hkv, int D,
                               int page_size, int max_pages, int num_pages, float scale, void* out, float* lse,
                               void* stream, void* workspace, size_t ws_bytes);

/* Workspace bytes mk_paged_attention needs (0 for invalid sizes). */
size_t mk_paged_attention_workspace_size(int B, int Hq, int Hkv);

/* Weight types of mk_moe_ffn_decode. */
enum { MK_WEIGHT_BF16 = 0, MK_WEIGHT_E4M3 = 1 };

/* The whole gated expert layer for a few tokens (a decode step), in one
 * kernel: routing and gates as points 1 and 2 above, then
 *   h(t,j) = silu(x[t,:] . W1[e]) * (x[t,:] . W3[e])  for the j-th expert e,
 *   out[t,:] = sum_j gate[t,j] * (h(t,j) . W2[e]),  j in order, without the
 *   experts whose logit is -inf: their weights are not read.
 * With MK_WEIGHT_BF16, x and the weights are bf16 and the scale pointers
 * NULL; h is carried with 16 significant bits.  With MK_WEIGHT_E4M3 they are
 * e4m3 with scales: a weight stands for its value times the scale of its
 * 128 x 128 block, x[t,c] for its value times x_scale[t, c/128] (what
 * mk_add_rmsnorm writes); h is rounded to e4m3 likewise, per row and 128
 * columns with the scale max |h| / 448 (1 where that maximum is below
 * 2^-100), before its product.
 *   x[T,H], logits[T,E] f32, W1[E,H,F], W3[E,H,F], W2[E,F,H],
 *   x_scale[T,H/128] f32, W1_scale[E,H/128,F/128] f32, W3_scale likewise,
 *   W2_scale[E,F/128,H/128] f32                                   -- read only
 *   out[T,H] bf16, overlapping no input                           -- written
 * Limits: 0 <= T <= 128, 1 <= k <= min(E, 8), E <= 256, H and F multiples of
 * 64 (bf16) or 128 (e4m3) up to 32768; x, weights and out 16-byte aligned,
 * f32 arrays 4.  Only the chosen experts' weights are read: once for
 * every 64 rows (or fewer) that choose the expert.
 * workspace: NULL (library cache) or mk_moe_ffn_decode_workspace_size()
 * bytes, 256-byte aligned, zero-filled before its first use and used by this
 * entry point only (with any sizes); one stream at a time.  The kernel's CTAs
 * wait for one another within bounds (2 s; then MK_ERR_TIMEOUT from
 * mk_get_status()). */
mk_status_t mk_moe_ffn_decode(const void* x, const float* x_scale, const float* logits, int T, int H, int E, int k,
                              const void* W1, const void* W3, const void* W2, const float* W1_scale,
                              const float* W3_scale, const float* W2_scale, int F, int weights, void* out,
                              void* stream, void* workspace, size_t ws_bytes);

/* Workspace bytes mk_moe_ffn_decode needs (0 for invalid sizes). */
size_t mk_moe_ffn_decode_workspace_size(int T, int H, int F, int E, int k, int weights);

/* ------------------------------------------------------------------------
 * Operators that fill, share and read a paged key-value cache.  Conventions as
 * for the operators of a decode step above.
 *
 * A cache of MK_CACHE_BF16 is what mk_paged_attention reads.  One of
 * MK_CACHE_FP4 holds of each row of D columns D/2 bytes, two e2m1 values each
 * (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign; the even column in the low half), and
 * beside them D/16 e4m3 scales, one per 16 columns: value * scale stands for
 * y / factor, with an optional fp32 factor per key-value head.  Quantized are
 *   scale = max(2^-9, e4m3(max |y / factor| / 6)),  value = e2m1(y / factor / scale),
 * to nearest, ties to even, limited to the types' largest values; a NaN among
 * the 16 makes them all NaN (by their scale).  72 bytes a row of 128 against 256. */
enum { MK_CACHE_NONE = 0, MK_CACHE_BF16 = 1, MK_CACHE_FP4 = 2 };

/* Pairs of columns that are rotated: i and i + rot/2, or 2i and 2i + 1. */
enum { MK_PAIR_HALVES = 0, MK_PAIR_NEIGHBOURS = 1 };

/* Arguments of mk_qk_norm_rope.  Strides of q, k and v in elements, of a cache
 * in its units (bf16 elements, or bytes), of its scales in bytes. */
typedef struct mk_qk_norm_rope {
    const void *q, *k, *v;            /* [T,Hq,D], [T,Hkv,D], [T,Hkv,D] bf16; v only with a cache */
    int64_t q_stride, q_head_stride;  /* between tokens, between heads */
    int64_t k_stride, k_head_stride;
    int64_t v_stride, v_head_stride;
    const void *q_weight, *k_weight;  /* [D] bf16, or NULL: not normalized */
    const int32_t* positions;         /* [axes,T] */
    int64_t position_stride;          /* between axes */
    const float* inv_freq;            /* [rot/2], finite */
    const uint8_t* pair_axis;         /* HOST [rot/2]: the axis of each pair; NULL: the first */
    void *q_out, *k_out, *v_out;      /* [T,Hq,D], [T,Hkv,D], [T,Hkv,D] bf16; see below */
    const int64_t* slots;             /* [T]: page * page_size + token in the page; negative: none */
    void *k_cache, *v_cache;
    int64_t page_stride, token_stride, head_stride;
    void *k_scales, *v_scales;        /* MK_CACHE_FP4 only */
    int64_t scale_page_stride, scale_token_stride, scale_head_stride;
    const float *k_factor, *v_factor; /* [Hkv], or NULL: 1; normal numbers, y / factor below 2^126 */
    int32_t T, Hq, Hkv, D, rot, axes, pairs, cache, page_size, num_pages;
    float eps;
    int32_t reserved;                 /* zero */
} mk_qk_norm_rope_t;

/* Norms of the queries' and keys' heads, their rotation by position, and the
 * way of keys and values into a cache, in one pass:
 *   y = x * rsqrt(mean(x^2) + eps) * weight      over a head's D columns,
 *   angle = positions[axis(i),t] * inv_freq[i]    for pair i of the first rot
 *   columns: (a, b) -> (a cos - b sin, b cos + a sin); the others pass.
 * A frequency is held in steps of 2^-64 of a turn, so the angle is exact to 2^-31 of a
 * turn for any position and frequencies up to 4; sines and cosines are then off by
 * 2^-21 of themselves, those of small angles and next to their zeros too (frequencies
 * of 2^-36 or more).  q_out gets the queries; k_out, if not NULL, the keys; with a cache, the keys and the values
 * (as they are) of token t go to slots[t], and with MK_CACHE_FP4 k_out and v_out
 * (both may be NULL) get what the cache holds of them.  Without a cache k_out is
 * needed, and v and v_out are not used.  A token with a negative slot is left
 * out of the cache; one with a slot past the pool too, and it is reported by
 * mk_get_status() (MK_ERR_DEVICE_FAULT).  The slots of a call must differ.
 * q_out may be q itself, and k_out k, where their rows lie one after the other;
 * no other outputs overlap inputs.
 * Limits: D and rot multiples of 16, D <= 256, rot <= D (0: no rotation), axes
 * <= 4, heads <= 65536; q, k, v, the weights and outputs 16-byte aligned with
 * strides of multiples of 8 elements; a bf16 cache likewise, a 4-bit cache
 * 4-byte aligned with strides of multiples of 4 bytes. */
mk_status_t mk_qk_norm_rope(const mk_qk_norm_rope_t* args, void* stream);

/* mk_paged_attention over a cache of MK_CACHE_FP4: the same formulas with
 *   k(j,c,:) = value * scale * k_factor[c],   v likewise with v_factor,
 * products and sums in fp32, except that the weights e^(s_j - m) enter the
 * product with v with 11 significant bits (those below 2^-24 of the largest
 * with fewer; below 2^-34 they count as 0 there), and q with its 8 relative to its head's
 * largest column (those below 2^-28 of that with fewer, to 2^-39 of it).  Element (page, token, head)
 * of a cache's values begins at byte page*page_stride + token*token_stride +
 * head*head_stride, D/2 bytes in a row; of its scales at page*scale_page_stride
 * + ..., D/16 bytes.  k and v share strides.  A cache whose rows of one head lie
 * side by side in a page is read fastest: D/16 bytes of scales are less than
 * the 32 that memory moves at a time.
 *   q[B,Hq,D] bf16 with q_stride elements between sequences, k_factor[Hkv] and
 *   v_factor[Hkv] f32 (may be NULL: 1), the others as above        -- read only
 * Limits as above, but: q 16-byte aligned and q_stride a multiple of 8; values
 * 16-byte aligned with strides of multiples of 16 bytes; scales D/16-byte
 * aligned with strides of multiples of D/16; fewer than 2^31 tiles of 16 keys
 * and 8 query heads in all; scale * k_factor[c] below 2^127.  A value's scale that is NaN
 * makes its columns of out NaN, a key's scale and an infinite or NaN query their heads'
 * out and lse.  Errors and lengths as above.
 * workspace: NULL (library cache) or mk_paged_attention_fp4_workspace_size()
 * bytes, 256-byte aligned, zero-filled before its first use and used by this
 * entry point only; one stream at a time. */
mk_status_t mk_paged_attention_fp4(const void* q, int64_t q_stride, const void* k_cache, const void* v_cache,
                                   int64_t page_stride, int64_t token_stride, int64_t head_stride, const void* k_scales,
                                   const void* v_scales, int64_t scale_page_stride, int64_t scale_token_stride,
                                   int64_t scale_head_stride, const float* k_factor, const float* v_factor,
                                   const int32_t* block_table, const int32_t* seq_lens, int B, int Hq, int Hkv, int D,
                                   int page_size, int max_pages, int num_pages, float scale, void* out, float* lse,
                                   void* stream, void* workspace, size_t ws_bytes);

/* Workspace bytes mk_paged_attention_fp4 needs (0 for invalid sizes). */
size_t mk_paged_attention_fp4_workspace_size(int B, int Hq, int Hkv);

/* Pages of a pool, shared between sequences.  The state is on the device:
 *   block_table[rows,max_pages] i32: row s holds the pages of sequence s, of
 *     which ceil(seq_lens[s] / page_size) count; entries behind them are
 *     neither read nor changed,
 *   seq_lens[rows] i32,
 *   refs[num_pages] i32: the rows that hold a page; 0: it is free.
 * Lists (parent, child, seqs, count: n entries, i32) are on the device too.  A
 * call whose list names a sequence outside the table, one sequence twice (a
 * parent may be), a count outside [0, most] or more room than a row has, or
 * that would need more pages than are free, changes nothing; mk_get_status()
 * then reports MK_ERR_DEVICE_FAULT.  An entry that is no page is left out, and
 * reported.  Results are whole numbers and the same for equal states.
 * Buffers: n_caches of them, each with num_pages pages of page_bytes[i] bytes,
 * page_strides[i] bytes apart, from caches[i] on (device); the three arrays are
 * HOST arrays, read before the call returns.  Pages move as fast as a copy where
 * addresses, strides and sizes are multiples of 16 bytes.
 * Limits: rows <= 65536, n <= 4096, max_pages*page_size < 2^31, num_pages <=
 * 2^30, page_bytes <= 2^31.  workspace: NULL (library cache) or
 * mk_pages_workspace_size(max_pages, num_pages, n) bytes, 256-byte aligned, of
 * any content; one stream at a time. */

/* Page src[i] to page dst[i], i < n, in every buffer.  The pages of dst differ,
 * and none of them is in src.  n has no limit here. */
mk_status_t mk_copy_pages(void* const* caches, const int64_t* page_strides, const int64_t* page_bytes, int n_caches,
                          int num_pages, const int32_t* src, const int32_t* dst, int n, void* stream);

/* Sequence child[i] gives its pages back and from now on holds those of
 * parent[i] as they were before the call, the last one, which may not be full,
 * among them (mk_extend_sequences copies it when one of them goes on).  A child
 * may be another's parent, or its own. */
mk_status_t mk_fork_sequences(int32_t* block_table, int32_t* seq_lens, int32_t* refs, int rows, int max_pages,
                              int num_pages, int page_size, const int32_t* parent, const int32_t* child, int n,
                              void* stream, void* workspace, size_t ws_bytes);

/* The sequences of the list give their pages back; their lengths become 0. */
mk_status_t mk_free_sequences(const int32_t* block_table, int32_t* seq_lens, int32_t* refs, int rows, int max_pages,
                              int num_pages, int page_size, const int32_t* seqs, int n, void* stream);

/* Room for count[i] <= most new tokens of sequence seqs[i], in the order of the
 * list: if its last page is not full and other rows hold it, those of the list
 * that were already given a copy not counted, it gets a copy of it (in every buffer); then
 * as many more pages as it needs.  New pages are the lowest free ones.
 * slots[n,most] i64 (may be NULL): the place of each new token, page *
 * page_size + token, -1 behind the last.  seq_lens counts the new tokens. */
mk_status_t mk_extend_sequences(int32_t* block_table, int32_t* seq_lens, int32_t* refs, int rows, int max_pages,
                                int num_pages, int page_size, const int32_t* seqs, const int32_t* count, int n, int most,
                                int64_t* slots, void* const* caches, const int64_t* page_strides,
                                const int64_t* page_bytes, int n_caches, void* stream, void* workspace, size_t ws_bytes);

/* The pages in use, `used` of them, become the first ones: the i-th one of
 * index >= used moves to the i-th free one below, in every buffer, and table_out
 * and refs_out (which may be block_table and refs) say so; the buffers' pages
 * from used on are then free. */
mk_status_t mk_compact_pages(const int32_t* block_table, const int32_t* seq_lens, const int32_t* refs, int rows,
                             int max_pages, int num_pages, int page_size, int32_t* table_out, int32_t* refs_out,
                             void* const* caches, const int64_t* page_strides, const int64_t* page_bytes, int n_caches,
                             void* stream, void* workspace, size_t ws_bytes);

/* Workspace bytes that mk_fork_sequences, mk_extend_sequences and (with n = 0)
 * mk_compact_pages need at most, whatever max_pages is; the other two take none.
 * 0 for invalid sizes. */
size_t mk_pages_workspace_size(int max_pages, int num_pages, int n);

/* Synchronise `stream`, then return and clear the device error word
 * (MK_ERR_TIMEOUT / MK_ERR_DEVICE_FAULT), or MK_ERR_CUDA if the stream holds
 * a CUDA error.  MK_OK when nothing was recorded. */
mk_status_t mk_get_status(void* stream);

/* Detail of the last recorded device error: site code and CTA (or -1). */
void mk_last_error_detail(int32_t* site, int32_t* cta, int32_t* info);

/* Facts about the last dispatch call on this thread (grid, role split,
 * launches); the operators of a decode step do not change them. */
void mk_last_launch_info(mk_launch_info_t* info);

/* Copy the phase stamps of the last traced call (cfg.trace = 1) made with
 * these sizes on `stream` to the host: up to n uint64 values, 16 per CTA
 * (%globaltimer ns; 0 = phase not reached).  `workspace` is the caller
 * workspace that call used, or NULL for the library cache of `stream`.
 * Synchronises `stream`.  Slots of the fused single-SM kernel: 0 CTA start,
 * 1 its routing chunks done, 2 routing barrier passed, 3 scan and scatter
 * done, 4 scatter barrier passed (dispatch CTAs), 5 gather done (dispatch
 * CTAs), 6 GEMM role start, 7 GEMM role end, 8 combine barrier passed,
 * 9 combine done, 10 first full stage reaches the tensor core, 11 last MMA
 * completed, 15 CTA exit. */
mk_status_t mk_read_trace(void* stream, const void* workspace, int T, int H, int E, int k, uint64_t* out,
                          size_t n);

/* Free the library's workspace cache on every device (synchronises), and
 * forget the device addresses mk_moe_dispatch_gemm_noalloc looked up.  Graphs
 * that hold calls with the library's workspace cannot be replayed after. */
void mk_release_workspace(void);

/* Static string for a status code. */
const char* mk_status_string(mk_status_t s);

/* Library ABI version (major * 100 + minor). */
int mk_version(void);

#ifdef __cplusplus
}
#endif
#endif /* MK_H */
