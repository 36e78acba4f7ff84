/*
 * fa.h -- C ABI of the GB300 (sm_103a) FlashAttention-2 backward library.
 *
 * Operation (FlashAttention-2 backward as described by boostr 0.1.0,
 * src/ops/cuda/attention/flash_bwd.rs, doc comment of
 * flash_attention_bwd_impl, "Two-step process"):
 *   step 1 (preprocess)  D_i   = sum_c dO_ic * O_ic              (fp32)
 *   step 2 (main)        P_ij  = exp(scale * <Q_i, K_j> - LSE_i)  (masked -> 0)
 *                        dV_j  = sum_i P_ij dO_i
 *                        dS_ij = P_ij * (<dO_i, V_j> - D_i)
 *                        dK_j  = scale * sum_i dS_ij Q_i
 *                        dQ_i  = scale * sum_j dS_ij K_j
 * dK and dV of a key/value head are summed over the H / H_kv query heads
 * that share it; query head h uses key/value head h / (H / H_kv).
 * Query i sits at key position p_i = i + (S_k - S_q) (bottom-right alignment).
 * Causal masking keeps key j for query i iff j <= p_i.  A sliding window of
 * size w > 0 (fa_bwd_ex / fa_fwd_ex; boostr autograd_attention.rs carries
 * window_size through FlashAttentionConfig into both passes, 0 = none) also
 * drops keys with p_i - j >= w and, when not causal, keys with j - p_i >= w:
 * a causal query sees its w most recent keys, itself included.
 *
 * Layouts (shape checks of flash_attention_bwd_impl in flash_bwd.rs and of
 * flash_attention_backward in rustytorch rtx-flash-metal-attention
 * backward.rs): every tensor is dense row-major,
 *   Q, O, dO, dQ : [B, H,    S_q, d]   element type `dtype`
 *   K, V, dK, dV : [B, H_kv, S_k, d]   element type `dtype`
 *   LSE, D       : [B, H,    S_q]      float32, natural-log log-sum-exp of
 *                                      the scaled scores (-inf for a row
 *                                      that sees no key)
 *
 * Pointers are DEVICE pointers unless an entry point says otherwise.  The
 * caller owns every buffer it passes; the library owns an internal workspace
 * (fp32 dQ accumulator, D and a padded copy of LSE) cached per
 * (device, stream) and released by fa_shutdown().  All calls are
 * asynchronous on `stream` (a cudaStream_t; NULL = legacy default stream):
 * they return after enqueueing, results are valid in stream order, inputs
 * are never modified and outputs are fully overwritten.
 *
 * Errors: every entry point returns an fa_status.  Argument errors are
 * detected on the host before anything is enqueued (FA_ERR_INVALID_ARG /
 * FA_ERR_UNSUPPORTED) and fa_last_error() then names the argument and the
 * reason, like the InvalidArgument { arg, reason } errors of flash_bwd.rs.
 * CUDA launch failures give FA_ERR_CUDA.  Device-side waits are bounded: a
 * kernel whose wait runs out records it in the workspace error word and
 * returns; fa_check_device(stream) reports it as FA_ERR_TIMEOUT.
 */
#ifndef FA_H_
#define FA_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { FA_F32 = 0, FA_F16 = 1, FA_BF16 = 2 } fa_dtype;

typedef enum {
    FA_OK = 0,
    FA_ERR_INVALID_ARG = 1, /* bad pointer, shape, dtype, scale or alignment */
    FA_ERR_UNSUPPORTED = 2, /* valid but not implemented (head dim not 32/64/96/128/256) */
    FA_ERR_CUDA = 3,        /* a CUDA runtime / driver call failed */
    FA_ERR_TIMEOUT = 4,     /* a device-side bounded wait ran out */
    FA_ERR_NOMEM = 5        /* workspace allocation failed */
} fa_status;

/*
 * fa_bwd -- full FlashAttention-2 backward: preprocess D, then dQ, dK, dV.
 *   dO, Q, O      : [B, H, S_q, d]  dtype, 16-byte aligned
 *   K, V          : [B, H_kv, S_k, d] dtype, 16-byte aligned
 *   LSE           : [B, H, S_q] float32, 4-byte aligned
 *   dQ            : [B, H, S_q, d]  dtype, written
 *   dK, dV        : [B, H_kv, S_k, d] dtype, written (rows no query sees get 0)
 *   B, H, H_kv, S_q, S_k > 0, H % H_kv == 0, d in {32, 64, 96, 128, 256}
 *   scale         : finite, > 0 (usually 1/sqrt(d))
 *   causal        : 0 or 1
 *   dtype         : fa_dtype (F32, F16, BF16); accumulation is fp32
 *   stream        : cudaStream_t
 * F16/BF16 run tcgen05 tensor-core kernels: one for d <= 128 (d = 32 and 96
 * on the d = 64 and 128 instances, the missing columns read as zeros), one
 * for d = 256 (64-key tiles, dK and dV accumulated transposed); F32 runs an
 * FFMA kernel.
 * dQ is reduced across key tiles with fp32 atomics, so dQ may differ in the
 * last bits between runs (flash_bwd.rs, "dQ must be zeroed -- backward uses
 * atomicAdd"); dK and dV are deterministic.  fa_bwd_ex(..., deterministic = 1)
 * makes dQ reproducible too.
 */
int fa_bwd(const void* dO, const void* Q, const void* K, const void* V, const void* O,
           const float* LSE, void* dQ, void* dK, void* dV, int B, int H, int H_kv, int S_q,
           int S_k, int d, float scale, int causal, int dtype, void* stream);

/*
 * fa_bwd_preprocess -- step 1 alone (flash_bwd.rs, "Step 1: Preprocessing --
 * compute D = rowsum(dO (.) O) per query position"):
 *   D[b, h, i] = sum_c dO[b, h, i, c] * O[b, h, i, c], accumulated in fp32.
 *   dO, O : [B, H, S_q, d] dtype, 16-byte aligned;  D : [B, H, S_q] float32.
 */
int fa_bwd_preprocess(const void* dO, const void* O, float* D, int B, int H, int S_q, int d,
                      int dtype, void* stream);

/*
 * fa_fwd -- attention forward helper producing the O and LSE the backward
 * consumes (boostr autograd_attention.rs, var_flash_attention saves
 * q, k, v, output, lse):  O_i = sum_j softmax_j(scale <Q_i, K_j>) V_j and
 * LSE_i = log sum_j exp(scale <Q_i, K_j>) over the visible keys.
 *   Q : [B, H, S_q, d], K, V : [B, H_kv, S_k, d], O : [B, H, S_q, d] dtype;
 *   LSE : [B, H, S_q] float32.  Rows that see no key get O = 0, LSE = -inf.
 * F16/BF16 run a tcgen05 tensor-core kernel (fp32 accumulation, online
 * softmax over 128-key tiles, 64-key tiles at d = 256); F32 runs an FFMA
 * kernel.
 */
int fa_fwd(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H,
           int H_kv, int S_q, int S_k, int d, float scale, int causal, int dtype, void* stream);

/*
 * fa_bwd_ex / fa_fwd_ex -- fa_bwd / fa_fwd with the remaining arguments of the
 * pages' flash_attention_bwd / flash_attention_fwd calls (boostr
 * autograd_attention.rs, FlashAttentionBackward::backward and
 * var_flash_attention):
 *   window_size   : >= 0; 0 = no window, else the band described at the top.
 *                   Key tiles outside the band are skipped, not just masked.
 *                   A negative value gives FA_ERR_INVALID_ARG.
 *   deterministic : 0 = dQ reduced with fp32 atomics (as fa_bwd; the pages'
 *                   atomicAdd accumulation), bits may vary between runs;
 *                   1 = bitwise reproducible dQ: F16/BF16 add each 128x128
 *                   dQ tile's per-key-tile contributions in key-tile order
 *                   (the CTAs pass a turn counter in the workspace along; each
 *                   CTA takes its tile from a ticket counter in the order the
 *                   CTAs start and only ever waits for CTAs that started
 *                   before it, and every wait is bounded); F32 computes
 *                   dQ in its own kernel, each row summed over keys in index
 *                   order.  Other values give FA_ERR_INVALID_ARG.
 * dK and dV are bitwise reproducible in both modes.  Every other argument,
 * layout and result is that of fa_bwd / fa_fwd, which are these calls with
 * window_size = 0 and deterministic = 0.  The pages' backward rejects
 * window_size != 0; this library implements it.
 */
int fa_bwd_ex(const void* dO, const void* Q, const void* K, const void* V, const void* O,
              const float* LSE, void* dQ, void* dK, void* dV, int B, int H, int H_kv, int S_q,
              int S_k, int d, float scale, int causal, int window_size, int deterministic, int dtype,
              void* stream);
int fa_fwd_ex(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H,
              int H_kv, int S_q, int S_k, int d, float scale, int causal, int window_size, int dtype,
              void* stream);

/*
 * fa_bwd_host -- fa_bwd on HOST buffers (same arguments and layouts, every
 * pointer a host pointer; pinned memory gives full copy bandwidth and lets
 * copies overlap compute).  Copies the inputs to device buffers cached per
 * (device, stream), runs the backward on `stream`, copies dQ, dK, dV back and
 * returns once they are in the host buffers.  Problems with more than 32 MiB
 * of input are split into up to 4 chunks of whole (batch, kv head) units:
 * chunk c's inputs are copied on a library-owned stream while chunk c-1
 * computes on `stream` and chunk c-2's results are copied back on a second
 * library-owned stream.  Results are those of fa_bwd (dQ up to the order of
 * its fp32 reduction).
 */
int fa_bwd_host(const void* dO, const void* Q, const void* K, const void* V, const void* O,
                const float* LSE, void* dQ, void* dK, void* dV, int B, int H, int H_kv, int S_q,
                int S_k, int d, float scale, int causal, int dtype, void* stream);

/*
 * fa_bwd_noalloc -- fa_bwd for callers that cannot allocate device memory
 * (an allocator or memory pool that owns the GPU's memory, a host that must
 * not see the implicit synchronization of cudaMalloc / cudaFree, a runtime
 * that forbids libraries from allocating).  The pages have no counterpart of
 * this entry point.  Same arguments, layouts and results as fa_bwd; the
 * caller still passes every input and output buffer, and the library's
 * scratch comes from one fixed 32 MiB array compiled into the library, which
 * every GPU that loads the library holds until the process exits.
 *   * A shape needs 256 + 8*B*H*ceil(S_q/128)*128 + 4*B*H*S_q*d bytes of
 *     scratch (parts rounded up to 256 bytes); beyond 32 MiB the call returns
 *     FA_ERR_INVALID_ARG ("scratch: ...") and launches nothing.
 *   * The first call on a device looks the array's device address up and
 *     enqueues the clearing of its error words on `stream`: make that first
 *     call before any stream capture.
 *   * Every call shares the array (it keeps the last call's contents; each
 *     call re-zeroes what must start at zero).  Calls whose GPU work overlaps,
 *     e.g. on different streams, race: keep them in one stream's order.
 *   * The main kernel is the one fa_bwd would run for the same arguments.
 *   * Bounded-wait timeouts of this variant are recorded in the array and
 *     reported (then cleared) by fa_check_device(stream), as for fa_bwd.
 */
int fa_bwd_noalloc(const void* dO, const void* Q, const void* K, const void* V, const void* O,
                   const float* LSE, void* dQ, void* dK, void* dV, int B, int H, int H_kv,
                   int S_q, int S_k, int d, float scale, int causal, int dtype, void* stream);

/* Workspace bytes fa_bwd / fa_bwd_ex need for a shape (informational; the
 * library allocates and caches it itself): error words, padded LSE and D
 * copies, the fp32 dQ accumulator and the deterministic mode's turn counters. */
size_t fa_bwd_workspace_bytes(int B, int H, int S_q, int d);

/*
 * ---- Packed sequences and paged caches -----------------------------------
 *
 * Packed tensors hold N sequences of different lengths one after another, token
 * major: Q, O [T_q, H, d], K, V [T_k, H_kv, d]; sequence n owns query rows
 * [cu_q[n], cu_q[n+1]) and key rows [cu_k[n], cu_k[n+1]) (int32 device arrays
 * of N + 1 non-decreasing entries).  LSE is [H, T_q] float32.  Attention runs
 * inside each sequence, with the alignment, causal mask and window of fa_fwd_ex
 * for that sequence's S_q and S_k.  Sequences may be empty on either side: a
 * query that sees no key gets O = 0 and LSE = -inf; one whose visible scores hold
 * a NaN gets NaN in both, and in its gradients.  Nothing crosses from one sequence
 * to another; inside a sequence a hidden pair counts as weight 0 times its value, so
 * an infinite or NaN row of K or V may also show in rows that do not see it.  The
 * pages have no counterpart of these entry points.
 *
 *   strides    : element strides in host memory, or NULL for dense tensors; the
 *                head dimension itself is contiguous.  Every stride is > 0 and a
 *                multiple of 16 bytes, every tensor 16-byte aligned, so the
 *                slices of a joint QKV projection can be passed as they are.
 *   fill       : rows of no sequence (before cu_q[0], from cu_q[N] on) are
 *                0 = left as they were, 1 = set to O = 0 and LSE = -inf (every
 *                row, where the call computes nothing because of its lengths).
 *   workspace  : caller's scratch, 256-byte aligned, of at least the bytes that
 *                the matching *_workspace_bytes function gives.  It needs no
 *                initialisation and must not be shared by calls whose GPU work
 *                may overlap (graphs replayed side by side included).
 * All lengths are read on the device: no call synchronizes, and a captured call
 * replays with whatever lengths the arrays hold then.  Lengths that do not fit
 * the tensors (decreasing, negative, past T_q / T_k or 2^28 tokens) make the call
 * compute nothing; fa_check_device then reports FA_ERR_INVALID_ARG.
 * (fa_page_slots, whose outputs steer a cache, says below what it leaves then.)
 */

/*
 * fa_varlen_fwd -- attention forward over packed sequences.
 *   strides : {Q token, Q head, K token, K head, V token, V head, O token, O head}
 * F16/BF16 run a tcgen05 kernel (H / H_kv <= 128), F32 and wider head groups an
 * FFMA kernel.  The result is bitwise reproducible.
 */
int fa_varlen_fwd(const void* Q, const void* K, const void* V, void* O, float* LSE, const int* cu_q,
                  const int* cu_k, int N, int T_q, int T_k, int H, int H_kv, int d,
                  const long long* strides, float scale, int causal, int window_size, int fill,
                  int dtype, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes of fa_varlen_fwd (backward = 0) or fa_varlen_bwd (backward = 1);
 * 0 for arguments those calls refuse.  A backward's is 4 T_q H d bytes for dQ in fp32,
 * 1028 H for each 128-row tile of queries (T_q / 128 + N of them at most), 2048 d
 * (SMs + H_kv) at most for parts of long key tiles, and about 700 of plan per sequence. */
size_t fa_varlen_workspace_bytes(int N, int T_q, int T_k, int H, int H_kv, int d, int dtype,
                                 int backward);

/*
 * fa_varlen_bwd -- dQ, dK, dV of fa_varlen_fwd from dO, O and LSE (fa_bwd_ex inside
 * each sequence).  Rows of keys that no query sees get 0.
 *   strides       : {dO token, dO head, then the same of Q, K, V, O, dQ, dK, dV}
 *   deterministic : as in fa_bwd_ex (0 = dQ reduced with fp32 atomics, 1 =
 *                   bitwise reproducible dQ); dK and dV are reproducible in both
 *   fill          : gradient rows of no sequence are 0 = left, 1 = set to 0
 * F16/BF16 run tcgen05 kernels, F32 an FFMA kernel.
 */
int fa_varlen_bwd(const void* dO, const void* Q, const void* K, const void* V, const void* O,
                  const float* LSE, void* dQ, void* dK, void* dV, const int* cu_q, const int* cu_k,
                  int N, int T_q, int T_k, int H, int H_kv, int d, const long long* strides,
                  float scale, int causal, int window_size, int deterministic, int fill, int dtype,
                  void* workspace, size_t workspace_bytes, void* stream);

/*
 * fa_paged_fwd -- attention of each request's newest tokens over its pages of a
 * key/value cache (one token per request is a decode step, many a chunk of its
 * prompt; both kinds may share a call).
 *   K_cache, V_cache : [num_pages, page_size, H_kv, d], holding the new tokens too
 *   block_table      : [N, max_pages] int32 page numbers; entries behind a
 *                      request's last page are not read
 *   cu_q             : [N + 1] int32, the new tokens of request n are rows
 *                      [cu_q[n], cu_q[n+1]) of Q
 *   seq_lens         : [N] int32 tokens in the cache, the new ones included;
 *                      query i sits at position seq_lens[n] - S_q + i.  A request
 *                      longer than max_pages * page_size sees only the tokens that
 *                      its row of the table has room for; fa_check_device reports
 *                      it (FA_ERR_INVALID_ARG), the other requests are not touched
 *   strides          : {Q token, Q head, K page, K row, K head, V page, V row,
 *                      V head, O token, O head}
 * F16/BF16 caches whose page_size is a multiple of 8 that divides 128 or is a
 * multiple of 128 (64 at d = 256) run the tcgen05 kernel, others an FFMA kernel.
 * A table entry outside the cache reads as zeros and is reported by
 * fa_check_device (FA_ERR_INVALID_ARG).  With a window, pages that lie wholly
 * before it need not be valid any more.  The result is bitwise reproducible.
 */
int fa_paged_fwd(const void* Q, const void* K_cache, const void* V_cache, void* O, float* LSE,
                 const int* block_table, const int* cu_q, const int* seq_lens, int N, int T_q,
                 int num_pages, int page_size, int max_pages, int H, int H_kv, int d,
                 const long long* strides, float scale, int causal, int window_size, int fill,
                 int dtype, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes of fa_paged_fwd; 0 for arguments it refuses. */
size_t fa_paged_workspace_bytes(int N, int T_q, int H, int H_kv, int d, int page_size, int dtype);

/*
 * fa_page_slots -- pages and slots of a step's new tokens, on the device.
 *   ctx_lens    : [N] int32 tokens each request holds already
 *   cu_q        : [N + 1] int32 new tokens, as in fa_paged_fwd
 *   free_pages  : [num_free] int32 numbers of unused pages, taken from
 *                 free_start[0] on, in request order
 *   block_table : [N, max_pages] int32, in: the pages held; out: the new pages
 *                 behind them (other entries are left alone)
 *   slots       : [T] int64 out, page * page_size + row of each token; -1 for
 *                 rows of no request
 *   positions   : [T] int32 out, position of each token in its request, or -1
 *   seq_lens    : [N] int32 out, ctx_lens plus the new tokens
 *   free_next   : [1] int32 out, free_start[0] plus the pages taken (plus the pages
 *                 that the new tokens ask for, when the free list runs out)
 * When the free list or the table has no room, the entries and slots concerned
 * are -1 and fa_check_device reports FA_ERR_INVALID_ARG; a page that would stand
 * behind the table's last column is not taken.  Lengths that do not fit
 * (cu_q decreasing, negative or past T; ctx_lens negative or above 2^30) hand
 * nothing out: slots and positions are all -1, seq_lens is ctx_lens, free_next is
 * free_start[0], the table is left alone, and the check reports it.  The call changes
 * neither free_pages nor free_start, so running it again gives the same result;
 * an output that overlaps an input is refused.
 */
int fa_page_slots(const int* ctx_lens, const int* cu_q, const int* free_pages, const int* free_start,
                  int* block_table, long long* slots, int* positions, int* seq_lens, int* free_next,
                  int N, int T, int num_free, int page_size, int max_pages, void* stream);

/*
 * fa_paged_write -- K and V rows [T, H_kv, d] of new tokens to their slots of the
 * cache.  A negative slot is skipped; one past the cache is skipped and reported
 * by fa_check_device (FA_ERR_INVALID_ARG).  Slots must differ: of two rows with
 * the same slot either may be kept.
 *   strides : {K token, K head, V token, V head, K page, K row, K head of the
 *             cache, V page, V row, V head of the cache}
 */
int fa_paged_write(const void* K, const void* V, const long long* slots, void* K_cache, void* V_cache,
                   int T, int num_pages, int page_size, int H_kv, int d, const long long* strides,
                   int dtype, void* stream);

/* Synchronizes `stream`, then returns FA_ERR_TIMEOUT if a kernel of this
 * library on that stream, or an fa_bwd_noalloc call on this device, recorded
 * a bounded-wait timeout since the last check (clearing the record), else
 * FA_ERR_INVALID_ARG if a packed or paged call on this device was given lengths,
 * pages or slots that do not fit, else FA_OK (or FA_ERR_CUDA). */
int fa_check_device(void* stream);

/*
 * Per-kernel timing of fa_bwd calls (CUDA events recorded on the caller's
 * stream around each of the three launches: preprocess, main, dQ finalise).
 * fa_profile(1) clears the record and starts collecting, fa_profile(0)
 * stops.  fa_profile_read synchronizes on the recorded events and returns
 * the summed milliseconds per kernel in ms[0..2] and the number of fa_bwd
 * calls recorded.  Recording adds event records to the stream, nothing else.
 */
int fa_profile(int enable);
int fa_profile_read(float* ms, int* calls);

/*
 * fa_selftest_timeout -- failure-detection self-test (not needed in normal
 * use): launches on `stream` one CTA that waits, through the same bounded wait
 * the backward kernel uses, on a barrier nothing ever completes, with a limit
 * of `limit_ns` nanoseconds (0 < limit_ns <= 1e9).  The wait runs out and the
 * kernel records a timeout in the stream's workspace error word and returns;
 * fa_check_device(stream) then reports FA_ERR_TIMEOUT and the CUDA context
 * stays usable.  The bounded waits of the backward are the device side of the
 * pages' KernelError reporting (boostr flash_bwd.rs launch errors).
 */
int fa_selftest_timeout(unsigned long long limit_ns, void* stream);

/* Thread-local text of the last error ("arg: reason"); "" if none. */
const char* fa_last_error(void);

/* Frees every cached workspace of the calling process (all devices).  Must
 * not race with calls in flight. */
void fa_shutdown(void);

/* Library version string. */
const char* fa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FA_H_ */
