/*
 * attn.h — C ABI of the GB300 (sm_103a) fused attention library
 * (libattn_gb300.so).
 *
 * Operation.  Scaled-dot-product attention per (sequence, head):
 *     S = s * Q K^T,  P = softmax(S) row by row,  O = P V,
 * and its backward for the scalar loss whose gradient with respect to O is dO:
 *     dV = P^T dO,  dP = dO V^T,  dS = P ⊙ (dP - D),  D_i = sum_k dO_ik O_ik,
 *     dQ = s * dS K,  dK = s * dS^T Q.
 * Defined in "ops(8)：self-attention 的 CUDA 实现及优化 (下) - 深度分析",
 * §2.1 (forward, and the five backward steps with the softmax derivative) and
 * Appendix A; D is the row sum of dP ⊙ P that the softmax backward subtracts
 * (§2.1 step 3), computed from dO and O because the two are equal.  The
 * forward also returns the softmax statistic the backward needs (§1.3 of the
 * same page: "stats", only in training mode); here that is the natural-log
 * log-sum-exp of the scaled scores, LSE_i = ln sum_j exp(S_ij).
 * Causal masking: key j is visible to query i iff j <= i + (Tk - Tq): with
 * Tq == Tk that is the §2.2 CPU loop's t2 <= t; with fewer queries than keys
 * (separate query and key lengths, as the cuDNN graph of "ops(8)..." §1.3
 * allows) the queries are the last Tq positions of the key sequence
 * (bottom-right alignment).  Causal (or windowed) attention with more queries
 * than keys is not supported: Tq > Tk at fixed length, or a sequence with
 * Lq > Lk in a variable-length batch with separate offsets (attn_fwd_ex).
 *
 * Precision.  Inputs and outputs are bf16; products accumulate in fp32; the
 * softmax runs in fp32; P and dS are rounded to bf16 before they enter the
 * tensor-core products; dQ is accumulated across key tiles in fp32.
 *
 * Memory.  Every pointer is a DEVICE pointer except the offset tables
 * `cu_seqlens`, `cu_seqlens_q`, `cu_seqlens_k` (host) and the tensors of
 * attn_step_host (host).
 * The library allocates no device memory: the caller owns all buffers,
 * including the backward workspace, sized with attn_bwd_workspace_size().
 * Every tensor pointer must be 16-byte aligned.
 *
 * Layouts (`layout` argument):
 *   ATTN_LAYOUT_BTHD (0): q (B,Tq,H,dqk), k (B,Tk,H,dqk), v (B,Tk,H,dv),
 *       o and dO (B,Tq,H,dv); dq, dk, dv like q, k, v.
 *   ATTN_LAYOUT_PACKED_QKV (1): q, k, v point at slots 0, 1, 2 of one
 *       (B,T,3,H,d) buffer (k = q + H*d, v = q + 2*H*d elements), the format
 *       of "ops(8)..." §1.3 (QKV as (B, T, 3, NH, HS), no permute); o and dO
 *       are (B,T,H,d); dq, dk, dv likewise point at slots of a packed
 *       (B,T,3,H,d) gradient buffer.  Needs dqk == dv and Tq == Tk.
 *   Variable length: when `cu_seqlens` is non-NULL, B is the number of
 *       sequences, Tq == Tk is the TOTAL number of token rows, tensors are
 *       (Tq, H, d) (or (Tq, 3, H, d) packed), sequence b occupies rows
 *       cu_seqlens[b] .. cu_seqlens[b+1]-1 (int32, host memory, B+1 entries,
 *       cu_seqlens[0] == 0, nondecreasing, cu_seqlens[B] == Tq), and LSE is
 *       (H, Tq).  At most ATTN_MAX_VARLEN_SEQS sequences.  attn_fwd_ex /
 *       attn_bwd_ex also take separate key offsets (keys (Tk, H, d), Tk the
 *       total key count).
 *   Fixed length: LSE is (B, H, Tq) fp32.
 *
 * Supported head sizes: (dqk, dv) in {(64, 64), (128, 128), (192, 128)}.
 *
 * Errors.  Functions return ATTN_OK (0) or a negative ATTN_ERR_* code.
 * Argument errors are detected on the host before anything is launched.
 * Launches are asynchronous on `stream` (a cudaStream_t; NULL = the legacy
 * default stream); a device-side failure (a bounded wait inside a kernel that
 * gave up) is reported later through attn_fwd_status() / attn_bwd_status().
 *
 * Threading.  Calls on different streams with different workspaces may run
 * concurrently.  Calls that share a workspace must be ordered on the GPU.
 */
#ifndef ATTN_GB300_H
#define ATTN_GB300_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

#define ATTN_OK 0
#define ATTN_ERR_INVALID_ARG (-1)         /* NULL / misaligned pointer, bad size */
#define ATTN_ERR_UNSUPPORTED (-2)         /* head sizes, causal with Tq > Tk, ... */
#define ATTN_ERR_WORKSPACE_TOO_SMALL (-3) /* workspace_bytes below the query */
#define ATTN_ERR_CUDA (-4)                /* a CUDA runtime call or launch failed */
#define ATTN_ERR_TIMEOUT (-5)             /* a kernel's bounded wait gave up */
#define ATTN_ERR_INTERNAL (-6)            /* a kernel found its launch set-up unusable */
#define ATTN_ERR_SCRATCH_TOO_SMALL (-7)   /* attn_bwd_noalloc: problem exceeds its scratch */
#define ATTN_ERR_BAD_PAGE (-8)            /* a length or page index outside the paged cache */
#define ATTN_ERR_WORKSPACE_NOT_READY (-9) /* attn_decode: workspace was not initialised */

#define ATTN_LAYOUT_BTHD 0
#define ATTN_LAYOUT_PACKED_QKV 1
#define ATTN_MAX_VARLEN_SEQS 1024
#define ATTN_BLOCK 128 /* rows per block of a block-sparse mask (the kernels' tile) */

/*
 * Forward: O and (unless lse == NULL, inference mode) LSE.
 * q, k, v: inputs (bf16); o: output (bf16); lse: output (fp32) or NULL.
 * B, H, Tq, Tk, dqk, dv: sizes (see Layouts); causal: 0/1; scale: the s in
 * S = s Q K^T, finite and > 0 (the pages use 1/sqrt(dqk)); cu_seqlens: NULL or
 * host offsets.
 * Values that are not finite: a row that does not see a key of its sequence meets it
 * with a weight of zero wherever their tiles of 128 rows meet, so an infinity or a NaN
 * there can reach it.  Those of another sequence never reach it in the forward; in the
 * backward they can, where the two share a tile.
 * "ops(8)..." §1.2-1.3 (sdpa returns [O, stats]; stats only when training),
 * §2.1 forward formulas.
 */
int attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
             int Tq, int Tk, int dqk, int dv, int causal, float scale, const int* cu_seqlens,
             int layout, void* stream);

/*
 * Local (sliding-window) attention: as attn_fwd, with key j visible to query i
 * iff  i + (Tk - Tq) - window_left <= j <= i + (Tk - Tq) + window_right
 * (each bound >= 0, or -1 for no bound on that side; variable-length batches
 * use Tk - Tq = 0 within each sequence), intersected with the causal bound
 * when causal = 1.  (-1, -1) is attn_fwd; (-1, 0) is causal.  A window needs
 * Tq <= Tk.  A mask mode in the sense of "深度学习反向传播优化：2-CTA MMA模式与
 * 内存访问优化" §5.1-5.2 (FlexAttention-style variants as independent mask
 * modules): the kernels visit only the tiles the band touches and mask the
 * band's edge tiles per element.  Returns ATTN_ERR_INVALID_ARG for bounds
 * below -1.
 */
int attn_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                    int H, int Tq, int Tk, int dqk, int dv, int causal, int window_left,
                    int window_right, float scale, const int* cu_seqlens, int layout,
                    void* stream);

/*
 * Bytes of device workspace attn_bwd needs for these sizes (varlen: 1 when
 * cu_seqlens will be given; Tq is then the total token count).  The
 * workspace holds the fp32 dQ accumulator, D and LSE*log2(e) per query row,
 * one semaphore per (query tile, head), a work counter and a status word.
 * Returns 0 for invalid sizes.  "ops(8)..." §1.3: the caller-provided
 * workspace sized by a query, as the cuDNN graph does.
 */
size_t attn_bwd_workspace_size(int B, int H, int Tq, int Tk, int dqk, int dv, int varlen,
                               int deterministic);

/*
 * Backward: dq, dk, dv (bf16) from q, k, v, o, dO (bf16) and the forward's
 * lse (fp32, required).  deterministic = 1 adds each key tile's dQ
 * contribution in a fixed order (descending key tile, "深度学习反向传播优化：
 * 2-CTA MMA模式与内存访问优化" §3.2), so results are bit-identical run to run;
 * 0 uses unordered fp32 atomics (§3.1).  workspace: device memory of at least
 * attn_bwd_workspace_size() bytes, 256-byte aligned; its contents need no
 * initialisation.  "ops(8)..." §2.1 backward steps 1-5.
 */
int attn_bwd(const void* q, const void* k, const void* v, const void* o, const void* dO,
             const float* lse, void* dq, void* dk, void* dv_out, int B, int H, int Tq, int Tk,
             int dqk, int dv, int causal, float scale, const int* cu_seqlens, int layout,
             int deterministic, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Backward of attn_fwd_window (same window arguments; lse from that forward).
 * Keys that no query sees get dK = dV = 0.
 */
int attn_bwd_window(const void* q, const void* k, const void* v, const void* o, const void* dO,
                    const float* lse, void* dq, void* dk, void* dv_out, int B, int H, int Tq,
                    int Tk, int dqk, int dv, int causal, int window_left, int window_right,
                    float scale, const int* cu_seqlens, int layout, int deterministic,
                    void* workspace, size_t workspace_bytes, void* stream);

/*
 * The general forward: every option of the calls above in one entry point.
 *
 * Local window: as attn_fwd_window (window_left / window_right, -1 = open).
 *
 * Block-sparse attention: key j is visible to query i only where the block
 * mask marks the pair of blocks (i / ATTN_BLOCK, j / ATTN_BLOCK) with a
 * non-zero byte.  The block-sparse mask module of "深度学习反向传播优化：2-CTA
 * MMA模式与内存访问优化" §5.1-5.2 (FlexAttention and block-sparse variants built
 * from the same kernels by a mask module alone): the kernels skip every tile
 * pair the mask drops.
 *   block_mask: DEVICE pointer to uint8 [mask_batches][mask_heads][NQ][NK],
 *     C order, read only, owned by the caller, unchanged until the call's work
 *     on `stream` is done.  NQ = ceil(Tq / ATTN_BLOCK), NK = ceil(Tk /
 *     ATTN_BLOCK); for variable-length batches NQ = ceil(longest query
 *     sequence / ATTN_BLOCK), NK likewise for the keys, and sequence b uses its
 *     own block coordinates (entries past its ends are not read).
 *     mask_batches is 1 (one mask for every sequence) or B; mask_heads is 1 or
 *     H.  NULL: no block mask.
 * A query row that sees no key gets O = 0 and LSE = -inf (and, in attn_bwd_ex,
 * dQ = 0; it adds nothing to dK or dV).
 *
 * Variable-length batches with separate query and key lengths ("ops(8)..."
 * §1.3: seq_len_q and seq_len_kv given apart): cu_seqlens_q (host, B + 1
 * offsets into the (sum Tq, H, d) queries) and cu_seqlens_k (host, B + 1
 * offsets into the (sum Tk, H, d) keys and values); Tq and Tk are the totals.
 * cu_seqlens_k = NULL: the keys use cu_seqlens_q (Tq == Tk); both NULL: fixed
 * length.  Within sequence b the queries are the last Lq = cu_seqlens_q[b+1] -
 * cu_seqlens_q[b] of its Lk key positions (causal and windows align
 * bottom-right, as for fixed length); a causal or windowed sequence needs
 * Lq <= Lk (ATTN_ERR_UNSUPPORTED otherwise), and a sequence with queries needs
 * keys (ATTN_ERR_INVALID_ARG).  LSE is (H, sum Tq).  Packed QKV needs shared
 * offsets.
 *
 * Returns ATTN_ERR_INVALID_ARG for other mask_batches / mask_heads values or
 * offsets that do not start at 0, decrease, or do not end at the totals.
 */
int attn_fwd_ex(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                int Tq, int Tk, int dqk, int dv, int causal, int window_left, int window_right,
                const unsigned char* block_mask, int mask_batches, int mask_heads, float scale,
                const int* cu_seqlens_q, const int* cu_seqlens_k, int layout, void* stream);

/*
 * Backward of attn_fwd_ex (same options; lse from that forward).  Workspace as
 * for attn_bwd (its size query takes Tq = the total query count and varlen =
 * 1).  Deterministic mode adds the dQ contributions of the kept key tiles in
 * descending key-tile order.
 */
int attn_bwd_ex(const void* q, const void* k, const void* v, const void* o, const void* dO,
                const float* lse, void* dq, void* dk, void* dv_out, int B, int H, int Tq, int Tk,
                int dqk, int dv, int causal, int window_left, int window_right,
                const unsigned char* block_mask, int mask_batches, int mask_heads, float scale,
                const int* cu_seqlens_q, const int* cu_seqlens_k, int layout, int deterministic,
                void* workspace, size_t workspace_bytes, void* stream);

/*
 * Grouped heads: Hq query heads over Hk key heads, Hq a multiple of Hk; query
 * head h uses key head h / (Hq / Hk).  As attn_fwd_ex / attn_bwd_ex without a
 * block mask (causal, windows, variable length and what they refuse; Hq == Hk
 * is allowed), with the distances between token rows given tensor by tensor:
 * q, o, dO, dq (.., Hq, d), k, v, dk, dv (.., Hk, d), the heads of a row
 * adjacent, rows evenly spaced over the whole batch.  dk and dv are sums over
 * the group's query heads, accumulated in fp32 and rounded once.  LSE has Hq
 * heads.  No counterpart on the pages.
 * Values that are not finite: as in attn_fwd and attn_bwd (see there).
 * Workspace: attn_bwd_grouped_workspace_size() bytes (0 for invalid sizes):
 * that of attn_bwd for Hq heads, and, where there are few key tiles and heads,
 * the fp32 sums of parts of the groups.
 *
 * attn_rows: elements between token rows, a multiple of 8 and at least H*d (0:
 * dense, H*d); the slices of one projection (T, (Hq + 2 Hk) * d) have its
 * width.  NULL: all dense.  The forward reads q, k, v and o.
 */
typedef struct attn_rows {
  long long q, k, v, o, d_o, dq, dk, dv;
} attn_rows;
int attn_fwd_grouped(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                     int Hq, int Hk, int Tq, int Tk, int dqk, int dv, const attn_rows* rows,
                     int causal, int window_left, int window_right, float scale,
                     const int* cu_seqlens_q, const int* cu_seqlens_k, void* stream);
size_t attn_bwd_grouped_workspace_size(int B, int Hq, int Hk, int Tq, int Tk, int dqk, int dv,
                                       int varlen, int deterministic);
int attn_bwd_grouped(const void* q, const void* k, const void* v, const void* o, const void* dO,
                     const float* lse, void* dq, void* dk, void* dv_out, int B, int Hq, int Hk,
                     int Tq, int Tk, int dqk, int dv, const attn_rows* rows, int causal,
                     int window_left, int window_right, float scale, const int* cu_seqlens_q,
                     const int* cu_seqlens_k, int deterministic, void* workspace,
                     size_t workspace_bytes, void* stream);

/*
 * Backward for callers that cannot allocate device memory (a plugin whose host
 * framework owns all device memory, or a loop where a device-synchronising
 * cudaMalloc is not allowed).  Same arguments and results as attn_bwd, minus
 * the workspace: the library's own 32 MiB device array stands in for it, so
 * it needs attn_bwd_workspace_size() <= 32 MiB (larger problems return
 * ATTN_ERR_SCRATCH_TOO_SMALL; e.g. B=8, H=12, T=1024, d=64 fits).  The first
 * call in each CUDA context looks up the array's address (make it before any
 * stream capture); a call after the device's context was reset and
 * re-created looks it up again.  Every device that loads this code holds the
 * array until exit.  All calls share the array: calls that overlap on the GPU
 * race, so order them on one stream.  A device-side timeout of the last call
 * is read with attn_bwd_noalloc_status().  No counterpart on the pages.
 */
int attn_bwd_noalloc(const void* q, const void* k, const void* v, const void* o, const void* dO,
                     const float* lse, void* dq, void* dk, void* dv_out, int B, int H, int Tq,
                     int Tk, int dqk, int dv, int causal, float scale, const int* cu_seqlens,
                     int layout, int deterministic, void* stream);

/*
 * Synchronises `stream` and returns the device status of the last
 * attn_bwd_noalloc call on the current device (ATTN_OK or ATTN_ERR_TIMEOUT),
 * read from the library's scratch array; allocates nothing.  No counterpart
 * on the pages.
 */
int attn_bwd_noalloc_status(void* stream);

/*
 * Synchronises `stream` and returns the device status of the last backward
 * that used `workspace` (ATTN_OK or ATTN_ERR_TIMEOUT).
 */
int attn_bwd_status(const void* workspace, void* stream);

/*
 * Synchronises `stream`, returns the sticky device status of the forward
 * kernels on the current device (ATTN_OK or ATTN_ERR_TIMEOUT) and clears it.
 */
int attn_fwd_status(void* stream);

/*
 * Instrumentation: when both are non-NULL (cudaEvent_t handles), every later
 * attn_bwd call records event_start on its stream just before the backward
 * main kernel and event_stop just after it, so the caller can time that
 * kernel alone.  Pass two NULLs to turn it off.  Returns ATTN_OK, or
 * ATTN_ERR_INVALID_ARG when only one is NULL.  Benchmark support; no
 * counterpart on the pages.
 */
int attn_profile_main_kernel(void* event_start, void* event_stop);

/*
 * Instrumentation, like attn_profile_main_kernel: when all four are non-NULL
 * (cudaEvent_t handles), every later attn_bwd call records pre_start and
 * pre_stop around its preprocess kernel (D and the per-row statistics) and
 * convert_start and convert_stop around its dQ conversion kernel.  Four NULLs
 * turn it off; a mix returns ATTN_ERR_INVALID_ARG.  Benchmark support (the
 * HBM rates of the two memory-bound kernels); no counterpart on the pages.
 */
int attn_profile_aux_kernels(void* pre_start, void* pre_stop, void* convert_start,
                             void* convert_stop);

/*
 * Which backward main kernel later calls use where both apply (dqk = dv = 128,
 * no block mask, no left window edge): 0 = the library's choice, 1 = one CTA
 * per key tile, 2 = CTA pairs (two key tiles per cluster of two CTAs, tcgen05
 * pair MMAs, dQ contracted over both tiles before its atomics; "深度学习反向传播
 * 优化：2-CTA MMA模式与内存访问优化" §2.1-2.2 and §3.1).  Both give results within
 * the same tolerance; deterministic mode is bit-identical run to run with
 * either, though not between them (the pair kernel adds dQ per pair of key
 * tiles).  Returns ATTN_ERR_INVALID_ARG for other values.  Tests and
 * benchmarks use it to run both kernels.
 */
int attn_debug_set_bwd_variant(int variant);

/*
 * Counters of the library's host-side cache (TMA tensor maps and the
 * schedule tables of variable-length batches, reused across calls with the
 * same pointers, shapes and options): out4[0] tensor maps encoded, out4[1]
 * tensor maps reused, out4[2] tables built, out4[3] tables reused, since the
 * library was loaded.  Returns ATTN_ERR_INVALID_ARG for NULL.  Test and
 * diagnostics support; the cache itself follows the build-once, run-many
 * graphs of "ops(8)..." §1.3.
 */
int attn_debug_cache_stats(long long* out4);

/*
 * Test hook (host-side fault injection; 0 = normal operation): every ordered
 * dQ wait of later deterministic attn_bwd calls in this process waits for a
 * semaphore value `bias` higher than the one that will come (a bias above the
 * number of key tiles can never be met), so the bounded wait gives up and
 * attn_bwd_status() reports ATTN_ERR_TIMEOUT.  The kernels
 * stop, free their tensor memory and leave the CUDA context usable.  No
 * counterpart on the pages (whose printed spin-wait, §3.2 of "深度学习反向传播
 * 优化：2-CTA MMA模式与内存访问优化", has no bound).
 */
int attn_debug_set_wait_bias(int bias);

/*
 * Forward + backward for tensors in HOST memory, with the copies overlapped
 * with the kernels (the step a caller makes when its data starts and ends on
 * the host).  q, k, v, dO: host (B,T,H,d) bf16 inputs (layout 0, fixed
 * length, Tq == Tk == T); dq, dk, dv_out: host (B,T,H,d) bf16 outputs; o: host
 * (B,T,H,dv) bf16 output or NULL (O stays on the device).  Host memory should
 * be page-locked (cudaHostAlloc / cudaHostRegister): pageable memory works but
 * its copies do not overlap.  The heads are split into groups of at most
 * heads_per_group (0 = half the heads, rounded up); the first and the last
 * group are about half that size, to shorten the pipeline's fill and drain
 * (H = 16 with the default gives groups of 4, 8, 4).  Each group's slices are copied
 * in on h2d_stream, computed with attn_fwd + attn_bwd on `stream`, and copied
 * back on d2h_stream, two groups in flight.  With stream2 != NULL the two
 * alternating device sets compute on `stream` and stream2, so one group's
 * kernels can start on SMs that the previous group's last work items leave
 * idle.  NULL streams mean `stream` (no overlap).  scratch: device memory of at least
 * attn_step_host_scratch_size() bytes, 256-byte aligned, used only by this
 * call until `stream` passes its end.  Asynchronous: `stream` waits for every
 * copy, so synchronising `stream` makes the host outputs valid.  Results are
 * those of attn_fwd / attn_bwd on the whole tensors (bit-identical with
 * deterministic = 1).  No counterpart on the pages; it moves the data of the
 * step that "ops(8)..." §2.1 defines.
 */
size_t attn_step_host_scratch_size(int B, int H, int T, int dqk, int dv, int heads_per_group,
                                   int deterministic);
int attn_step_host(const void* q, const void* k, const void* v, const void* dO, void* o,
                   void* dq, void* dk, void* dv_out, int B, int H, int T, int dqk, int dv,
                   int causal, float scale, int deterministic, int heads_per_group,
                   void* scratch, size_t scratch_bytes, void* stream, void* stream2,
                   void* h2d_stream, void* d2h_stream);

/*
 * Synchronises `stream` and returns the device status of the last
 * attn_step_host call that used `scratch` with these sizes: ATTN_OK, or the
 * first group's ATTN_ERR_TIMEOUT (forward or backward).
 */
int attn_step_host_status(const void* scratch, int B, int H, int T, int dqk, int dv,
                          int heads_per_group, int deterministic, void* stream);

/*
 * Position rotation and the paged key / value cache: what a model needs around
 * the attention above to see positions (training and serving) and to generate
 * token by token (serving).  No counterpart on the pages.  As with the calls
 * above, make the first call on a device before any stream capture.
 */

/*
 * The rotation of a head's columns begin .. begin + dim - 1, in pairs (a, b):
 * at position p pair i turns by the angle p * w_i,
 *     a' = a cos(p w_i) - b sin(p w_i),   b' = a sin(p w_i) + b cos(p w_i);
 * the other columns pass unchanged.  style: which columns form pair i,
 * ATTN_ROPE_HALVES: (begin + i, begin + dim/2 + i); ATTN_ROPE_PAIRS:
 * (begin + 2i, begin + 2i + 1).  begin and dim are multiples of 16 (dim > 0).
 * rates: DEVICE array of dim/2 words from attn_rope_rates(); 8-byte aligned.
 */
#define ATTN_ROPE_HALVES 0
#define ATTN_ROPE_PAIRS 1
typedef struct attn_rotation {
  const unsigned long long* rates;
  int begin, dim, style;
} attn_rotation;

/*
 * Host helper (no GPU needed): converts n angular rates w_i (radians per
 * position, finite, of any size) to the fixed-point form that the kernels
 * read: the fraction of a turn per position, times 2^64.  A position times
 * that word, modulo 2^64, is the angle modulo one turn, so an angle is as exact
 * at position two billion as at position one (the word is off by at most two
 * units and 2^-105 of the rate).  Copy the words to the device once.  Returns
 * ATTN_ERR_INVALID_ARG for NULL, n <= 0 or a rate that is not finite.
 */
int attn_rope_rates(const double* rates_rad, int n, unsigned long long* out);

/*
 * Rotates q and k by their positions: q (B,Tq,Hq,d) and k (B,Tk,Hk,d) bf16
 * into q_out and k_out.  Either of q and k may be NULL (with its output); an
 * output may be its input (in place), and must not overlap it otherwise.
 * Positions are those of attn_fwd: key j of a sequence is at pos0 + j, query
 * i at pos0 + i + (Tk - Tq) (pass Tk = Tq when only q is given and its
 * positions start at pos0; Tk = 0 is taken where k is NULL, Tq = 0 where q is).  Variable length: cu_seqlens_q / cu_seqlens_k as in
 * attn_fwd_ex (host; Tq and Tk are then totals, at most ATTN_MAX_VARLEN_SEQS
 * sequences), sequence by sequence.  A query in front of the first key
 * (Lq > Lk) has a negative position, which turns the other way.  *_row: elements
 * between token rows of each tensor, a multiple of 8 and at least H*d (0: H*d); a
 * slot of a packed (B,T,3,H,d) buffer has 3*H*d.  inverse = 1 turns the other way: the gradient
 * with respect to the unrotated tensor from the gradient with respect to the
 * rotated one.  d is 64, 128 or 192; pos0 >= 0 and every position below 2^31.
 * Computed in fp32 and rounded to bf16 once.
 */
int attn_rope(const void* q, const void* k, void* q_out, void* k_out, int B, int Hq, int Hk,
              int Tq, int Tk, int d, long long q_row, long long k_row, long long q_out_row,
              long long k_out_row, const attn_rotation* rotation, int inverse, int pos0,
              const int* cu_seqlens_q, const int* cu_seqlens_k, void* stream);

/*
 * Norm of each query and key head, with the position rotation in the same pass:
 *     y = R(p) (x / sqrt(mean x^2 + eps) * w)
 * over the d columns of a head; w: device fp32 per column, shared by the heads (q_weight,
 * k_weight; 4-byte aligned; NULL: ones), R(p) the rotation at the row's position.
 * eps: positive, normal and finite.  rotation may be NULL (the norm alone).  Tensors,
 * rows, positions, offsets and limits are those of attn_rope; an output may be its
 * input.  Computed in fp32 and rounded to bf16 once.
 *
 * attn_norm_rope_bwd: from x (q, k as the forward had them) and the gradients dq_out,
 * dk_out of the forward's outputs, the gradients dq, dk of q and k (which may be
 * dq_out / dk_out or q / k themselves, and must not overlap them otherwise) and,
 * where not NULL, those of the weights (fp32, d values each, written, not added to):
 * sums over all rows and heads in fp32, in a fixed order, so that they have the same
 * bits every run.  Either of q and k may be NULL with all that goes with it.
 * attn_norm_rows: elements between token rows of each (0: dense); NULL: all dense.
 * workspace: attn_norm_rope_bwd_workspace_size(d) bytes (0 for another d), 256-byte
 * aligned; needs no initialisation.  Calls that share it must be ordered on the GPU.
 */
typedef struct attn_head_norm {
  const float* q_weight;
  const float* k_weight;
  float eps;
} attn_head_norm;
typedef struct attn_norm_rows {
  long long q, k, dq_out, dk_out, dq, dk;
} attn_norm_rows;
int attn_norm_rope(const void* q, const void* k, void* q_out, void* k_out, int B, int Hq, int Hk,
                   int Tq, int Tk, int d, long long q_row, long long k_row, long long q_out_row,
                   long long k_out_row, const attn_head_norm* norm, const attn_rotation* rotation,
                   int pos0, const int* cu_seqlens_q, const int* cu_seqlens_k, void* stream);
size_t attn_norm_rope_bwd_workspace_size(int d);
int attn_norm_rope_bwd(const void* q, const void* k, const void* dq_out, const void* dk_out,
                       void* dq, void* dk, float* dq_weight, float* dk_weight, int B, int Hq,
                       int Hk, int Tq, int Tk, int d, const attn_norm_rows* rows,
                       const attn_head_norm* norm, const attn_rotation* rotation, int pos0,
                       const int* cu_seqlens_q, const int* cu_seqlens_k, void* workspace,
                       size_t workspace_bytes, void* stream);

/*
 * A paged cache of keys and values.  k and v (device) hold num_pages pages of
 * page_size tokens for each of `heads` key heads, dqk and dv columns wide;
 * element (page, token, head, c) of k is at page * k_page_stride + token *
 * k_token_stride + head * k_head_stride + c, in elements (v likewise), so
 * (pages, tokens, heads, d), (pages, heads, tokens, d) and one buffer that
 * holds both k and v are all described by strides.  Bases and strides are
 * multiples of 16 bytes.  To be appended to, rows must have their own memory, and
 * each stride be as long as all that the shorter ones cover (else
 * ATTN_ERR_INVALID_ARG); the decode only reads, and takes any.
 * type ATTN_CACHE_BF16: bf16.  ATTN_CACHE_E4M3: 8-bit floats, each standing
 * for its value times k_scale[head] / v_scale[head] (device fp32, one value
 * per key head, from 2^-100 to 2^100; NULL: 1).
 *
 * Which pages a sequence uses is in its row of a block table (device int32,
 * B rows of max_pages entries, table_stride entries apart): its token t is
 * token t % page_size of page table[t / page_size].  Entries past a sequence's
 * length are not read.
 *
 * lens (device int32, B): the number of tokens of each sequence INCLUDING the
 * ones that this step appends.  The same array serves attn_cache_append and
 * attn_decode of one step.  A length of 0 marks an unused row.
 *
 * A device-side error (a length that exceeds max_pages * page_size, a page
 * index outside 0 .. num_pages - 1) faults nothing: such tokens are not written
 * and not attended, and attn_cache_status() reports ATTN_ERR_BAD_PAGE.
 */
#define ATTN_CACHE_BF16 0
#define ATTN_CACHE_E4M3 1
typedef struct attn_paged_cache {
  void* k;
  void* v;
  const float* k_scale;
  const float* v_scale;
  long long k_page_stride, k_token_stride, k_head_stride;
  long long v_page_stride, v_token_stride, v_head_stride;
  int type, num_pages, page_size, heads, dqk, dv;
} attn_paged_cache;

/*
 * Appends new tokens to the cache: k (T,heads,dqk) and v (T,heads,dv) bf16,
 * rows k_row and v_row elements apart (multiple of 8; 0: dense).  Without
 * cu_seqlens every sequence brings T / B tokens (T a multiple of B); with it
 * (host, B + 1 offsets, as in attn_fwd) sequence b brings rows cu_seqlens[b] ..
 * cu_seqlens[b+1] - 1.  The i-th of n new tokens of sequence b takes position
 * lens[b] - n + i; a token whose position is negative (an unused row) is
 * ignored, and nothing of it is written.
 * rotation: NULL, or the rotation applied to k on the way (at the token's
 * position).  q, q_out: NULL, or the same tokens' queries (T,Hq,dqk) bf16, rows
 * q_row / q_out_row elements apart, rotated into q_out (in place if equal;
 * copied without a rotation).
 * e4m3 caches keep x / scale rounded to nearest even and saturated at +-448
 * (NaN stays NaN).  Two new tokens must not fall on the same cache slot.
 */
int attn_cache_append(const attn_paged_cache* cache, const int* block_table, int max_pages,
                      long long table_stride, const int* lens, int B, int T,
                      const int* cu_seqlens, const void* k, long long k_row, const void* v,
                      long long v_row, const void* q, long long q_row, void* q_out,
                      long long q_out_row, int Hq, const attn_rotation* rotation, void* stream);

/*
 * attn_cache_append with the norm of attn_norm_rope on the way: k and q are normed (each with
 * its weight) and then turned; v is not.  norm NULL: attn_cache_append.
 */
int attn_cache_append_norm(const attn_paged_cache* cache, const int* block_table, int max_pages,
                           long long table_stride, const int* lens, int B, int T,
                           const int* cu_seqlens, const void* k, long long k_row, const void* v,
                           long long v_row, const void* q, long long q_row, void* q_out,
                           long long q_out_row, int Hq, const attn_head_norm* norm,
                           const attn_rotation* rotation, void* stream);

/*
 * Attention of one new token per sequence over the cache: q (B,Hq,dqk) bf16
 * (rows q_row elements apart; 0: dense), o (B,Hq,dv) bf16, lse (B,Hq) fp32 or
 * NULL.  Query head h uses key head h / (Hq / heads); Hq is a multiple of
 * `heads`.  scale: positive, normal and below 2^127.  The token sits at position
 * lens[b] - 1 and sees the keys 0 .. lens[b] - 1, or with window_left >= 0 only
 * lens[b] - 1 - window_left .. lens[b] - 1 (-1: no window).  A row that sees no
 * key (lens[b] <= 0), or whose scores are all -inf, gets O = 0 and LSE = -inf.
 * Keys and values that a row does not see never touch it, whatever their bits;
 * one that it sees and that is not finite makes the row not finite (a key whose
 * score is -inf weighs nothing), and so does a largest score beyond fp32.
 *
 * The work is split over the keys of all sequences alike, in pieces that depend
 * on the lengths alone; the parts of a row are joined by the last of its CTAs to
 * finish, in a fixed order: results do not depend on timing (they do on the
 * pieces, so on the other lengths of the batch).
 *
 * workspace: attn_decode_workspace_size() bytes, 256-byte aligned, initialised
 * ONCE with attn_decode_workspace_init() before its first use; each call
 * leaves it ready for the next, of any sizes.  Calls that share a workspace,
 * captured graphs included, must be ordered on the GPU.  A workspace that was
 * not initialised writes nothing, and attn_cache_status() reports
 * ATTN_ERR_WORKSPACE_NOT_READY.
 */
size_t attn_decode_workspace_size(void);
int attn_decode_workspace_init(void* workspace, size_t workspace_bytes, void* stream);
int attn_decode(const attn_paged_cache* cache, const int* block_table, int max_pages,
                long long table_stride, const int* lens, int B, const void* q, long long q_row,
                void* o, float* lse, int Hq, int window_left, float scale, void* workspace,
                size_t workspace_bytes, void* stream);

/*
 * Attention of a chunk of new tokens per sequence over the cache, which holds
 * them already: a prompt's next piece, a few drafted tokens, single tokens, in
 * one batch.  q (T,Hq,dqk) bf16, rows q_row elements apart; without cu_seqlens
 * every sequence brings T / B tokens (T a multiple of B), with it (host, B + 1
 * offsets, B at most ATTN_MAX_VARLEN_SEQS) sequence b brings rows cu_seqlens[b]
 * .. cu_seqlens[b+1] - 1, as in attn_cache_append.  o (T,Hq,dv) bf16, lse
 * (T,Hq) fp32 or NULL, dense.  Query head h uses key head h / (Hq / heads); Hq
 * is a multiple of `heads`, at most 128 times it.  The i-th of n new tokens sits
 * at position p = lens[b] - n + i and sees the keys 0 .. p, or with window_left
 * >= 0 only p - window_left .. p.  scale: as in attn_decode.
 * A row that sees no key (p < 0), or whose scores are all -inf, gets O = 0 and
 * LSE = -inf.  As in attn_decode, keys and values that a row does not see never
 * touch it, whatever their bits, one that it sees and that is not finite makes the
 * row not finite (a key whose score is -inf weighs nothing, but its value has to
 * be finite), and so does a largest score beyond fp32.
 * Weights enter the second product rounded to bf16 (their sum is of unrounded
 * ones): O is off by at most 2^-8 of the sum of |w_j v_j| besides its own
 * rounding.  Over an e4m3 cache the operands are fp16: each row of queries times
 * a power of two, exact but for elements below 2^-28 of the row's largest, and
 * weights of 11 bits down to 2^-21 of the largest so far, zero below 2^-32.
 *
 * The work is cut into equal shares of key tiles, at places that depend on the
 * lengths alone, and parts of a row are joined in a fixed order by a second
 * launch: results do not depend on timing (they do on the other lengths of the
 * batch).
 *
 * workspace: attn_prefill_workspace_size() bytes, 256-byte aligned; needs no
 * initialisation and keeps nothing between calls.  Calls that share a workspace,
 * captured graphs included, must be ordered on the GPU.
 */
size_t attn_prefill_workspace_size(void);
int attn_prefill(const attn_paged_cache* cache, const int* block_table, int max_pages,
                 long long table_stride, const int* lens, int B, int T, const int* cu_seqlens,
                 const void* q, long long q_row, void* o, float* lse, int Hq, int window_left,
                 float scale, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Synchronises `stream`, returns the sticky device status of attn_cache_append,
 * attn_decode and attn_prefill on the current device (ATTN_OK, ATTN_ERR_BAD_PAGE,
 * ATTN_ERR_WORKSPACE_NOT_READY or ATTN_ERR_TIMEOUT, a bounded wait that gave up; the
 * first since the last read) and clears it, in one step: what a call on another stream
 * reports meanwhile is kept for the next read.
 */
int attn_cache_status(void* stream);

/* Static text for an ATTN_* code. */
const char* attn_strerror(int code);

/*
 * Host helper (no GPU needed): the order in which the kernels take the
 * sequences of a variable-length batch — longest first, ties by index
 * ("深度学习反向传播优化..." §3.2, batches sorted by expected time).
 * Writes `nseq` sequence indices to order_out.  Returns ATTN_OK or
 * ATTN_ERR_INVALID_ARG.
 */
int attn_varlen_order(const int* cu_seqlens, int nseq, int* order_out);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_GB300_H */
