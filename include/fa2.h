/*
 * fa2.h -- C ABI of libfa2.so: FlashAttention-2 exact multi-head attention,
 * forward and backward, on one sm_103a (GB300) GPU.
 *
 * The operation (sources: the FlashAttention-2 write-ups
 *   "FlashAttention学习笔记(2)" (amentiraz.github.io), sections "V2 的运作流程"
 *       and "V2中的thread blocks排布";
 *   "大猿搬砖简记" (damodev.csdn.net), the V2 forward / backward walk-throughs;
 *   "flash-attention123和ring-attention" (blog.csdn.net), 优化1 - 优化4):
 *
 *   for every batch b and head h, with S = scale * Q K^T (N x N):
 *     causal: S[i][j] = -inf for j > i   (top-left alignment, key j visible to query i iff j <= i)
 *     O   = softmax_rows(S) V
 *     L_i = ln(sum_j exp(S[i][j]))       (the logsumexp; the only softmax statistic stored)
 *   backward, given dO:
 *     P = exp(S - L), dV = P^T dO, dP = dO V^T, D_i = sum_c dO[i][c] * O[i][c],
 *     dS = P o (dP - D), dQ = scale * dS K, dK = scale * dS^T Q.
 *
 * Layout of every tensor argument: contiguous row-major [B][H][N][d] of 16-bit
 * floats (dtype FA2_FP16 or FA2_BF16); lse is contiguous fp32 [B][H][N].
 * Q, K and V share the sequence length N (self-attention), except in
 * fa2_fwd_qk / fa2_bwd_qk, where K and V have their own length Nk.
 *
 * Ownership: the caller allocates and owns every buffer, including the
 * backward workspace. The library keeps only a per-device status word (a
 * static device variable) and never frees caller memory.
 *
 * Execution: every compute entry point only enqueues work on `stream` (a
 * cudaStream_t, or NULL for the legacy default stream) and returns; nothing
 * synchronises the host. Outputs are fully overwritten, never accumulated into,
 * and must not overlap any input.
 *
 * Errors: every entry point returns an fa2_status (int). Arguments are checked
 * before anything is launched; on an error nothing is launched and no output
 * is touched. A kernel never traps: a bounded wait that runs out writes
 * FA2_ERR_DEVICE_TIMEOUT into the device status word, and a value in device
 * memory that a paged-cache kernel cannot follow writes FA2_ERR_PAGE;
 * fa2_get_device_status() reports them.
 */
#ifndef FA2_H_
#define FA2_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum fa2_status {
  FA2_OK = 0,
  FA2_ERR_INVALID_ARG = 1,    /* null pointer, B/H/N < 1, bad dtype/causal, scale not finite or <= 0 */
  FA2_ERR_UNSUPPORTED = 2,    /* d not in {64, 128}, or a size beyond the documented limits */
  FA2_ERR_ALIGNMENT = 3,      /* a tensor pointer not 16-byte aligned (lse: 4-byte; workspace: 256-byte) */
  FA2_ERR_ARCH = 4,           /* current device is not compute capability 10.3 (sm_103) */
  FA2_ERR_CUDA = 5,           /* a CUDA runtime / driver call or kernel launch failed */
  FA2_ERR_DEVICE_TIMEOUT = 6, /* a kernel gave up on a bounded wait (see fa2_get_device_status) */
  FA2_ERR_WORKSPACE = 7,      /* backward workspace missing or smaller than fa2_bwd_workspace_size */
  FA2_ERR_OVERLAP = 8,        /* an output buffer overlaps an input buffer */
  FA2_ERR_PAGE = 9            /* device status only: a paged-cache call met a page number, a length or a
                                 count outside the cache (see "Paged key-value cache") */
} fa2_status;

/* FA2_FP32: the norm weights of fa2_rotary_fwd and fa2_rotary_bwd only. */
typedef enum fa2_dtype { FA2_FP16 = 0, FA2_BF16 = 1, FA2_FP32 = 2 } fa2_dtype;

/* Forward pass (FlashAttention-2 forward: Q rows outer, K/V tiles inner, online
 * softmax with running max m and sum l, one division by l at the end, only
 * L = m + ln l stored; fully masked causal K/V tiles skipped).
 *   q, k, v : device, [B][H][N][d] dtype, 16-byte aligned, read only.
 *   o       : device, [B][H][N][d] dtype, 16-byte aligned, written.
 *   lse     : device, [B][H][N] fp32, 4-byte aligned, written (natural log).
 *   B, H, N : >= 1; B <= 65535, H <= 65535, B*H*N < 2^31.
 *   d       : 64 or 128.
 *   causal  : 0 or 1.
 *   scale   : finite, > 0 (usually 1/sqrt(d)).
 *   dtype   : FA2_FP16 or FA2_BF16 (q, k, v, o share it).
 *   stream  : cudaStream_t or NULL. */
int fa2_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int N,
            int d, int causal, float scale, int dtype, void* stream);

/* K/V-split forward ("大猿搬砖简记", thread-block section: when the (row block,
 * batch, head) workers cannot fill the SMs, each worker's K/V range may be cut
 * into num_splits parts run by separate blocks, whose partial results are then
 * combined to recover the global softmax). num_splits is the part count of the
 * longest worker (n_max K/V tiles of 128 keys); a worker with n tiles (shorter
 * under the causal mask) gets min(n, ceil(n * num_splits / n_max)) balanced,
 * contiguous, non-empty parts. A worker with one part writes O and L itself;
 * the parts of the others write fp32 O / l and logsumexp into the workspace
 * and count their arrival per 128-row tile; the part that arrives last forms
 * L = ln sum_s exp(lse_s), O = sum_s exp(lse_s - L) O_s (no CTA waits on
 * another; the counters are zeroed on the stream before the launch). Blocks
 * are launched longest row block first, heads varying fastest.
 * Same result as fa2_fwd up to rounding.
 *   num_splits : 1 .. 128 (1 runs fa2_fwd and ignores the workspace).
 *   workspace  : device, >= fa2_fwd_split_workspace_size(...) bytes, 256-byte
 *                aligned, scratch owned by the caller (contents ignored on
 *                entry, undefined on exit).
 *   other arguments as in fa2_fwd. */
int fa2_fwd_split(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                  int N, int d, int causal, float scale, int dtype, int num_splits, void* workspace,
                  size_t workspace_bytes, void* stream);

/* Forward pass in the FlashAttention-1 loop order, for measuring the loop
 * order ("FlashAttention学习笔记(2)", the FlashAttention-1 forward algorithm
 * and the comparison of the two loop orders): K/V blocks outer, query blocks
 * inner, one CTA per (batch, head). At every (K/V block j, query block i) step
 * the running O_i (kept normalised), row max m_i and row sum l_i are read from
 * and written back to the workspace in HBM:
 *   m_new = max(m_i, m~), l_new = e^(m_i - m_new) l_i + e^(m~ - m_new) l~,
 *   O_i <- (l_i e^(m_i - m_new) O_i + e^(m~ - m_new) P~ V_j) / l_new,
 * with m~, P~ = exp(S - m~), l~ of the block S = scale Q_i K_j^T. The same
 * O and L as fa2_fwd up to rounding. Query and key lengths are equal.
 *   workspace : device, >= fa2_fwd_kv_outer_workspace_size(...) bytes,
 *               256-byte aligned, scratch owned by the caller (contents
 *               ignored on entry, undefined on exit).
 *   other arguments as in fa2_fwd. */
int fa2_fwd_kv_outer(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                     int N, int d, int causal, float scale, int dtype, void* workspace,
                     size_t workspace_bytes, void* stream);

/* Bytes of workspace fa2_fwd_kv_outer needs: B*H x N x (d + 2) fp32 (O_i, m_i,
 * l_i), each array rounded up to 256 bytes. Returns 0 for invalid sizes. */
size_t fa2_fwd_kv_outer_workspace_size(int B, int H, int N, int d);

/* One forward + backward step on HOST buffers: q, k, v, dO are read from host
 * memory and o, lse, dq, dk, dv written back to host memory, the copies
 * overlapped with the kernels. Every (batch, head) is independent
 * ("FlashAttention学习笔记(2)", V2中的thread blocks排布), so the B*H heads are
 * cut into chunks of heads_per_chunk consecutive heads and pipelined on three
 * internal streams: upload of chunk c+1, fa2_fwd + fa2_bwd of chunk c,
 * download of chunk c-1, with two device slots. The results are the bits of
 * fa2_fwd + fa2_bwd on device copies of the same tensors.
 *   q, k, v, dO       : host, [B][H][N][d] dtype, read only. Pinned
 *                       (page-locked) memory lets the copies overlap.
 *   o, dq, dk, dv     : host, [B][H][N][d] dtype, written.
 *   lse               : host, [B][H][N] fp32, written.
 *   heads_per_chunk   : >= 1, or 0 for ceil(B*H / 8).
 *   workspace         : device, >= fa2_step_host_workspace_size(...) bytes,
 *                       256-byte aligned, owned by the caller.
 *   stream            : a stream of the current device (or NULL). The chain
 *                       starts after the work queued on it and the stream
 *                       waits for the chain's end; host buffers must stay
 *                       valid until then. Calls on one device are enqueued
 *                       one at a time (a per-device lock).
 *   other arguments as in fa2_fwd. */
int fa2_step_host(const void* q, const void* k, const void* v, const void* dO, void* o, float* lse,
                  void* dq, void* dk, void* dv, int B, int H, int N, int d, int causal, float scale,
                  int dtype, int heads_per_chunk, void* workspace, size_t workspace_bytes,
                  void* stream);

/* Device workspace fa2_step_host needs: two slots, each of 8 [hc][N][d]
 * 16-bit tensors, one [hc][N] fp32 tensor and fa2_bwd's workspace for one
 * chunk (hc = heads per chunk as above); each array rounded up to 256 bytes.
 * Returns 0 for invalid sizes. */
size_t fa2_step_host_workspace_size(int B, int H, int N, int d, int heads_per_chunk);

/* Bytes of workspace fa2_fwd_split needs: num_splits x B*H x N x (d + 1) fp32
 * (the parts' O / l and logsumexp) plus B*H x ceil(N / 256) x 2 int32 arrival
 * counters, each of the three arrays rounded up to 256 bytes. Returns 0 for
 * invalid sizes. */
size_t fa2_fwd_split_workspace_size(int B, int H, int N, int d, int num_splits);

/* The split count of the same page: for each candidate s in 1 .. min(128,
 * num_sms, K/V tiles of the longest worker), the SM utilisation of the split
 * launch; returns the smallest s whose utilisation is at least 0.95 of the
 * best. The page does not define utilisation; here it is the fraction of the
 * SMs' time spent on K/V tiles, useful tiles / (num_sms * makespan), when the
 * launch's CTAs (row blocks of 256 queries longest first, each block's parts
 * in order, heads fastest) start in launch order on the SM that frees first,
 * each taking its K/V tiles plus 1 tile of fixed cost, plus 6 more if its row
 * block is split (partial write and merge) -- costs measured on GB300. 1 when
 * the unsplit launch already reaches 0.95. To split automatically, a caller
 * passes this count (with the device's SM count) to fa2_fwd_split; forward()
 * of the Python binding does so by default. Host only; results are cached
 * per shape. Returns 0 for invalid arguments. */
int fa2_num_splits(int B, int H, int N, int d, int causal, int num_sms);

/* Forward with different query and key lengths: q, o [B][H][Nq][d], lse
 * [B][H][Nq]; k, v [B][H][Nk][d]. The pages keep seqlen_q and seqlen_k
 * distinct ("FlashAttention学习笔记(2)", V2中的thread blocks排布) without stating
 * the causal mask for unequal lengths; here it is top-left: key j is visible
 * to query i iff j <= i, so query i sees keys 0 .. min(i, Nk - 1). Keys past
 * Nk are masked. Other arguments and limits as in fa2_fwd (for Nq and Nk). */
int fa2_fwd_qk(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
               int Nq, int Nk, int d, int causal, float scale, int dtype, void* stream);

/* Bytes of device workspace fa2_bwd needs: the fp32 row sums D = rowsum(dO o O)
 * and L * log2(e), each [B*H][N rounded up to 128], then 256 bytes for the
 * work counter of the main launch. Returns 0 for invalid sizes. */
size_t fa2_bwd_workspace_size(int B, int H, int N, int d);

/* Backward pass (FlashAttention-2 backward: D = rowsum(dO o O) first; then K/V
 * column blocks outer, Q tiles inner, S and P recomputed from L, dK/dV
 * accumulated on chip; dQ, which accumulates along the key direction, in fp32
 * on chip by a query-tile worker of its own -- no atomics, bit-reproducible).
 *   q, k, v, o, dO : device [B][H][N][d] dtype, 16-byte aligned (o and lse from fa2_fwd).
 *   lse            : device [B][H][N] fp32.
 *   dq, dk, dv     : device [B][H][N][d] dtype, 16-byte aligned, written.
 *   workspace      : device, >= fa2_bwd_workspace_size(B,H,N,d) bytes, 256-byte
 *                    aligned, scratch owned by the caller; contents on entry
 *                    are ignored and on exit undefined.
 *   other arguments as in fa2_fwd. */
int fa2_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse,
            const void* dO, void* dq, void* dk, void* dv, int B, int H, int N, int d, int causal,
            float scale, int dtype, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of device workspace fa2_bwd_atomic needs: fa2_bwd's, then the fp32 dQ
 * accumulator [B*H][N rounded up to 128][d]. Returns 0 for invalid sizes. */
size_t fa2_bwd_atomic_workspace_size(int B, int H, int N, int d);

/* The same gradients as fa2_bwd, computed the way the pages' column workers
 * do it ("FlashAttention学习笔记(2)", Foward和backward中的thread block划分; "大猿
 * 搬砖简记", V2 backward): one CTA per 128-key column block keeps K_j, V_j in
 * shared memory and dK_j, dV_j in TMEM while the query tiles stream past, and
 * adds each dQ_i contribution (dS K, fp32) into an accumulator in global
 * memory with TMA reduce-adds; the preprocessing pass zeroes the accumulator
 * and a last pass writes dq = scale * accumulator. Five products per (key
 * block, query tile) pair, against seven for fa2_bwd, but on GB300 it runs
 * slower than fa2_bwd (the reduce-adds and the longer per-tile chain of the
 * compute warps); kept as the measured alternative. The order of the
 * reduce-adds varies from run to run, so dq is not bit-reproducible (dk and
 * dv are). Equal query and key lengths.
 *   workspace : >= fa2_bwd_atomic_workspace_size(B,H,N,d) bytes, 256-byte aligned.
 *   other arguments as in fa2_bwd. */
int fa2_bwd_atomic(const void* q, const void* k, const void* v, const void* o, const float* lse,
                   const void* dO, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                   int causal, float scale, int dtype, void* workspace, size_t workspace_bytes,
                   void* stream);

/* Backward with different query and key lengths (mask as in fa2_fwd_qk): q, o,
 * dO, dq [B][H][Nq][d], lse [B][H][Nq]; k, v, dk, dv [B][H][Nk][d]. Keys that
 * no query sees (causal, Nk > Nq) get dk = dv = 0. The workspace is
 * fa2_bwd_workspace_size(B, H, Nq, d) bytes. Other arguments as in fa2_bwd. */
int fa2_bwd_qk(const void* q, const void* k, const void* v, const void* o, const float* lse,
               const void* dO, void* dq, void* dk, void* dv, int B, int H, int Nq, int Nk, int d,
               int causal, float scale, int dtype, void* workspace, size_t workspace_bytes,
               void* stream);

/* fa2_bwd, plus: phase_events (4 cudaEvent_t created by the caller, or NULL)
 * are recorded on `stream` before the preprocessing kernel, between it and
 * the main launch (the dK/dV and dQ workers), and twice after the main launch,
 * so the caller can time the two launches. */
int fa2_bwd_timed(const void* q, const void* k, const void* v, const void* o, const float* lse,
                  const void* dO, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                  int causal, float scale, int dtype, void* workspace, size_t workspace_bytes,
                  void* const* phase_events, void* stream);

/* fa2_bwd_atomic with the same four phase events: before the preprocessing
 * kernel, between it and the column workers' launch, between that and the dq
 * conversion, and after it. */
int fa2_bwd_atomic_timed(const void* q, const void* k, const void* v, const void* o,
                         const float* lse, const void* dO, void* dq, void* dk, void* dv, int B,
                         int H, int N, int d, int causal, float scale, int dtype, void* workspace,
                         size_t workspace_bytes, void* const* phase_events, void* stream);

/* fa2_bwd without a caller-provided workspace, for callers that must not
 * allocate device memory: code running inside a memory pool or a framework
 * allocator it does not own, or a process that fixes its device footprint at
 * start-up and may not call cudaMalloc afterwards. (The FlashAttention-2 pages
 * have no counterpart to this entry point; it is a property of this library.)
 * The backward's scratch -- the row sums D and L*log2(e), 8 bytes per query
 * row with rows padded to 128 per head, and a 256-byte work counter -- lives
 * in a 16 MiB + 256 byte array built into
 * the library, one per GPU that loads it, held until the process exits. Its
 * gradients are the bits of fa2_bwd on the same inputs.
 *   arguments  : as fa2_bwd, minus the workspace.
 *   limit      : fa2_bwd_workspace_size(B,H,N,d) <= 16 MiB + 256 (for example up to
 *                B*H = 256 heads of N = 8192); larger sizes return
 *                FA2_ERR_UNSUPPORTED and touch nothing.
 *   set-up     : the first call on a device looks up the array's device
 *                address with that device current and keeps it for the life
 *                of the process; make that first call before any stream
 *                capture. A device reset (cudaDeviceReset) reloads the
 *                library's device code at a new address, so do not use this
 *                entry point (or the library's status word) across a reset.
 *   concurrency: every call on a device shares the one array, so calls that
 *                may overlap on the GPU (different streams, or different host
 *                threads) race on it; serialise them. Nothing needs clearing
 *                between calls: each call writes every scratch entry it reads.
 *   allocation : none (no cudaMalloc, cudaFree or allocating library call). */
int fa2_bwd_noalloc(const void* q, const void* k, const void* v, const void* o, const float* lse,
                    const void* dO, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                    int causal, float scale, int dtype, void* stream);

/* ---- Paged key-value cache ------------------------------------------------
 * Generation after a prompt: the keys and values of earlier tokens live in a
 * cache of pages, a new token attends to them, and a cache that may not grow
 * is cut back by the attention weight that its tokens have gathered.
 *
 *   k_cache, v_cache : device [num_pages][Hkv][page_size][d] dtype, 16-byte
 *                      aligned. Any page_size >= 1.
 *   table            : device int32 [B][max_pages]: the pages of each sequence.
 *                      Slot j of sequence b lies in page table[b][j / page_size].
 *                      Entries past the slots in use are not read.
 *   lens             : device int32 [B]: slots in use, 0 .. L, with
 *                      L = max_pages * page_size.
 *   weights          : device fp32 [B][Hkv][L]: the attention weight gathered by
 *                      the token of each slot. They belong to the sequence, not
 *                      to the page: sequences may share the pages of a common
 *                      prefix and still be counted apart.
 *   positions        : device int32 [B][Hkv][L]: the position in the text of the
 *                      token of each slot (after an eviction slots are in no
 *                      order, and each head has kept other tokens).
 *   d, dtype         : as in fa2_fwd. Query heads: Hq = g * Hkv, g <= 128; query
 *                      head x reads key head x / g. B, Hq, Hkv <= 65535;
 *                      B * Hkv < 2^27; num_pages * Hkv * page_size < 2^31;
 *                      L <= 2^30.
 *
 * Lengths, counts and pages are read on the device, so a captured graph follows
 * them. A page number outside 0 .. num_pages - 1 is not followed: its slots
 * count as masked (decode), are not written (append) or not moved (evict). A
 * length or count outside its range is cut to it. Either sets FA2_ERR_PAGE in
 * the device status word. */

/* Attention of one new token per sequence, whose own key and value are in the
 * cache (fa2_cache_append first):
 *   s_j = scale q . k_j for the slots j < lens[b], L = ln sum_j e^(s_j),
 *   o = sum_j e^(s_j - L) v_j;  lens[b] = 0: o = 0, L = -inf.
 * With weights (both or neither pointer):
 *   weights_out[j] = weights[j] + sum over the g query heads of e^(s_j - L)
 * for j < lens[b]; slots past that are left as they were.
 *   q, o        : device [B][Hq][d] dtype, 16-byte aligned; o is written.
 *   lse         : device [B][Hq] fp32, written.
 *   weights_out : may be weights itself.
 *   workspace   : device, >= fa2_paged_decode_workspace_size(...) bytes,
 *                 256-byte aligned, scratch owned by the caller.
 * P is not rounded before its product with V (fp16: to 2^-21 of itself), so o
 * carries the rounding to dtype and errors of fp32's size. An infinite V entry of a
 * slot that weighs anything gives an infinite o. The cache is read once for each 16
 * query heads of a key head. The result does not depend on timing: repeated calls
 * give the same bits. */
int fa2_paged_decode(const void* q, const void* k_cache, const void* v_cache, const int* table,
                     const int* lens, const float* weights, float* weights_out, void* o, float* lse,
                     int B, int Hq, int Hkv, int d, int num_pages, int page_size, int max_pages,
                     float scale, int dtype, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace of fa2_paged_decode: the partial results of a fixed number of CTAs
 * and, with weights (nonzero), the fp32 logits [B][Hq][L]. 0 for invalid sizes. */
size_t fa2_paged_decode_workspace_size(int B, int Hq, int Hkv, int d, int page_size, int max_pages,
                                       int weights);

/* fa2_paged_decode (without weights) for sequences that begin with the same slots,
 * which are read and multiplied once for all of them. Sequence b has the prefix if
 * lens[b] >= prefix_len; its first prefix_len slots must then hold what the prefix's
 * slots hold (as a rule they are the same pages; the last one, where the prefix ends
 * inside a page, may be a copy). A shorter sequence is read by its own table alone.
 *   prefix      : device int32 [prefix_pages]: the prefix's pages, in order.
 *   prefix_len  : device int32 [1]: its slots, 0 .. prefix_pages * page_size (cut to
 *                 it, FA2_ERR_PAGE).
 *   prefix_pages: >= 1; prefix_pages * page_size <= 2^30.
 *   workspace   : device, >= fa2_prefix_decode_workspace_size(...) bytes, 256-byte
 *                 aligned, scratch owned by the caller.
 *   other arguments as in fa2_paged_decode.
 * Prefix slots past the last multiple of 16 (or of the largest power of two that
 * divides page_size, if that is less) are read for each sequence by its own table. In
 * the prefix P enters its product with a relative error of 2^-16 (bf16), or 2^-22 and
 * 2^-36 of the row's largest (fp16), or as in fa2_paged_decode where its kernel attends
 * to the prefix too, which goes by B * Hq / Hkv, Hkv, d and prefix_pages * page_size. An
 * infinite V entry gives what it gives in fa2_paged_decode; where that makes NaN of a
 * product in the prefix the call takes longer, about 0.13 us for each slot. The result
 * does not depend on timing: repeated calls give the same bits. */
int fa2_prefix_decode(const void* q, const void* k_cache, const void* v_cache, const int* table, const int* lens,
                      const int* prefix, const int* prefix_len, void* o, float* lse, int B, int Hq, int Hkv, int d,
                      int num_pages, int page_size, int max_pages, int prefix_pages, float scale, int dtype,
                      void* workspace, size_t workspace_bytes, void* stream);

/* Workspace of fa2_prefix_decode: the parts of the prefix, 256 fp32 rows of d for each
 * 256 query rows of a key head and each CTA, and of the own slots. 0 for invalid
 * sizes. */
size_t fa2_prefix_decode_workspace_size(int B, int Hq, int Hkv, int d, int page_size, int max_pages);

/* Appends new tokens: token i < num_new[b] of sequence b goes to slot
 * lens[b] + i; lens_out[b] = lens[b] + num_new[b]. Tokens past L are dropped
 * (FA2_ERR_PAGE).
 *   k, v        : device [B][Hkv][T][d] dtype, 16-byte aligned (a prompt as
 *                 fa2_fwd takes it, or T = 1).
 *   num_new     : device int32 [B], 0 .. T (a padded batch), or NULL: T each.
 *                 B * Hkv * T < 2^31.
 *   weights     : or NULL; the new slots get new_weights[B][Hkv][T] (fp32; for a
 *                 prompt, fa2_key_weights), or 0 if that is NULL.
 *   positions   : or NULL; the new slots get next_pos[b] + i (int32 [B]).
 *   lens_out    : device int32 [B], not lens itself.
 * Pages that several sequences name must not be appended to. */
int fa2_cache_append(const void* k, const void* v, void* k_cache, void* v_cache, const int* table,
                     const int* lens, const int* num_new, float* weights, const float* new_weights,
                     int* positions, const int* next_pos, int* lens_out, int B, int Hkv, int T, int d,
                     int num_pages, int page_size, int max_pages, int dtype, void* stream);

/* Eviction: every (sequence, key head) with lens[b] > budget keeps budget slots,
 * in place, in slots 0 .. budget - 1; lens_out[b] = min(lens[b], budget). Kept
 * are, in this order, recent tokens (position >= next_pos[b] - recent; without
 * positions the last `recent` slots) and those of the largest weight; NaN counts
 * as the smallest, -0 as 0; of equal ones the lower slot stays. Kept slots below
 * budget stay where they are; the i-th evicted slot below budget (ascending)
 * takes the row, weight and position of the i-th kept slot at or past it.
 * Pages past the new length may be given to other sequences afterwards.
 *   weights_out, positions_out : slots below lens_out[b] are written, the others
 *                 left as they were; each may be its input itself.
 *   positions, positions_out, next_pos : all or none. next_pos[b] is the
 *                 position that the next token will get.
 *   budget      : >= 1.  recent: 0 .. budget. With M = min(budget, L - budget):
 *                 B * Hkv * ceil(M / 64) < 2^31.
 *   lens_out    : device int32 [B], not lens itself.
 *   workspace   : device, >= fa2_cache_evict_workspace_size(...) bytes,
 *                 256-byte aligned, scratch owned by the caller.
 * Pages that several sequences name must not be evicted from. After
 * FA2_ERR_PAGE the contents of the sequence concerned are undefined. */
int fa2_cache_evict(void* k_cache, void* v_cache, const int* table, const int* lens, const float* weights,
                    float* weights_out, const int* positions, int* positions_out, const int* next_pos,
                    int* lens_out, int B, int Hkv, int d, int num_pages, int page_size, int max_pages,
                    int budget, int recent, int dtype, void* workspace, size_t workspace_bytes,
                    void* stream);

/* Workspace of fa2_cache_evict: per (sequence, key head) two int32 lists of at
 * most min(budget, L - budget) moves and their count. 0 for invalid sizes. */
size_t fa2_cache_evict_workspace_size(int B, int Hkv, int page_size, int max_pages, int budget);

/* Page tables brought from one set of lengths to another, in place: new requests
 * (lens[b] = 0), growth, eviction and the end of a sequence (new_lens[b] = 0) alike.
 * A sequence has the pages table[b][i], i < ceil(length / page_size).
 *   Pages past the new length are given back: refs[page] falls by one, and a page
 *   whose count reaches 0 goes to the free list. Then each sequence that grows takes
 *   the pages it lacks from the end of the list, sequences in order; taken pages get
 *   the count 1. The first sequence for which the list does not suffice, and all that
 *   grow by pages after it, get none and keep their length. The pages that are freed
 *   go to the list in reverse order of (sequence, page index) - of several releases of
 *   one page the last counts - so that undoing a resize restores the list.
 *   table       : device int32 [B][max_pages]; entries past a length are left as they
 *                 were.
 *   lens, new_lens : device int32 [B], 0 .. L (cut to it, FA2_ERR_PAGE).
 *   refs        : device int32 [num_pages]: how many sequences name each page; 0: it is
 *                 in the free list. A program that shares a page adds to its count.
 *   free_pages  : device int32 [num_pages], num_free: device int32 [1]: the free list
 *                 is free_pages[0 .. num_free - 1].
 *   lens_out    : device int32 [B]: new_lens[b], or lens[b] where the pages did not
 *                 suffice. Not lens or new_lens.
 *   workspace   : device, >= fa2_cache_resize_workspace_size(...) bytes, 256-byte
 *                 aligned, scratch owned by the caller.
 * B * max_pages <= 2^31 - 2^14. A page number that the cache does not have, or a page
 * given back more often than it was named, is not freed and sets FA2_ERR_PAGE; the pool's
 * contents are then undefined (but stay within it). Repeated calls give the same
 * bits. */
int fa2_cache_resize(int* table, const int* lens, const int* new_lens, int* refs, int* free_pages, int* num_free,
                     int* lens_out, int B, int num_pages, int page_size, int max_pages, void* workspace,
                     size_t workspace_bytes, void* stream);

/* Workspace of fa2_cache_resize; 0 for invalid sizes. */
size_t fa2_cache_resize_workspace_size(int B, int num_pages, int page_size, int max_pages);

/* Accumulated attention weight of a prompt's keys, after fa2_fwd / fa2_fwd_qk:
 *   out[b][h][j] = sum over the g = Hq / Hkv query heads x of key head h and the
 *   queries i < q_lens[b] that see key j of e^(scale q_i . k_j - lse_i).
 *   q           : device [B][Hq][N][d] dtype; lse: device fp32 [B][Hq][N], the
 *                 forward's (over keys repeated g times where g > 1).
 *   k           : device [B][Hkv][Nk][d] dtype.
 *   q_lens      : device int32 [B], 0 .. N (cut to it), or NULL: N each. A causal
 *                 batch padded on the right counts only its real queries, and
 *                 padded keys get 0; padded rows of q, k and lse may hold anything.
 *   out         : device fp32 [B][Hkv][Nk], written.
 *   causal      : top-left, as in fa2_fwd_qk. Keys that no query sees get 0.
 *   workspace   : device, >= fa2_key_weights_workspace_size() bytes, 256-byte
 *                 aligned, scratch owned by the caller.
 * Sizes as in fa2_fwd, g <= 128. Repeated calls give the same bits. */
int fa2_key_weights(const void* q, const void* k, const float* lse, const int* q_lens, float* out, int B,
                    int Hq, int Hkv, int N, int Nk, int d, int causal, float scale, int dtype,
                    void* workspace, size_t workspace_bytes, void* stream);

size_t fa2_key_weights_workspace_size(void);

/* ---- Rotary positions -------------------------------------------------------
 * Queries and keys turned by their positions, as attention expects them, from a
 * projection's output in its own layout; with weights, each head's row is normed
 * first, in the same pass. For a row x of d elements at position p:
 *   n = (mean(x^2) + eps)^(-1/2),  u_i = x_i n weight_i     (no weights: u = x)
 *   y_a = amplitude (u_a cos t - u_b sin t),  y_b = amplitude (u_b cos t + u_a sin t),
 *   t = p freqs[j]
 * for the pairs j < rotary_dim / 2, with (a, b) = (j, j + rotary_dim / 2), or
 * (2j, 2j + 1) if interleaved; y_i = u_i for i >= rotary_dim. Sums and products are fp32.
 * An angle is formed to 2^-31 turns at any position, for frequencies up to 2^40, and
 * rounded to 24 bits (at most 2^-26 turns) for its sine and cosine. y is rounded once.
 * The sum of squares of a row has to be finite in fp32.
 *   q, k          : device [B][Hq][N][d], [B][Hk][N][d] dtype, rows of d contiguous
 *                   elements, 16-byte aligned, other strides below. k may be NULL
 *                   (Hk = 0, and nothing that belongs to it).
 *   freqs         : device fp64 [rotary_dim / 2], radians per position, finite.
 *   positions     : device int32; position_mode 0: NULL, token i of every sequence is
 *                   at position i; 1: [B], at positions[b] + i; 2: [B][N]. Positions
 *                   fit in 31 bits and a sign.
 *   q_weight, k_weight : device [d] of weight_dtype (dtype or FA2_FP32), 16-byte
 *                   aligned; both (k_weight with k) or neither.
 *   q_out, k_out  : like q and k, written. Their rows must not overlap, nor anything
 *                   that is read; q_out and k_out may be heads side by side in one
 *                   buffer.
 *   strides       : host, 12 element strides: batch, head and token of q, k, q_out and
 *                   k_out; >= 0, multiples of 8 (that of a dimension of size 1 is not
 *                   used). An input's stride may be 0.
 *   rotary_dim    : a multiple of 16, 16 .. d.   d: 64 or 128.   eps: >= 0.
 *   limits        : B, Hq, Hk <= 65535; B * N * (ceil(Hq / 4) + ceil(Hk / 4)) < 2^31. */
int fa2_rotary_fwd(const void* q, const void* k, const double* freqs, const int* positions, const void* q_weight,
                   const void* k_weight, void* q_out, void* k_out, const long long* strides, int B, int Hq, int Hk,
                   int N, int d, int rotary_dim, int position_mode, int interleaved, float eps, float amplitude,
                   int dtype, int weight_dtype, void* stream);

/* Gradients of fa2_rotary_fwd. With g the gradient of y turned back by -t (and
 * amplitude), per row
 *   weight_grad_i = sum over rows of g_i x_i n,
 *   x_grad_i = n (weight_i g_i - x_i n mean_k(weight_k g_k x_k n));  no weights: x_grad = g.
 *   dq, dk           : gradients of q_out and k_out.
 *   q, k             : the forward's inputs; NULL without weights.
 *   q_grad, k_grad   : written; layout rules of q_out and k_out.
 *   q_weight_grad, k_weight_grad : device [d] of weight_dtype, written; with weights.
 *   strides          : host, 18: of dq, dk, q, k, q_grad and k_grad.
 *   workspace        : device, >= fa2_rotary_bwd_workspace_size(...) bytes, 256-byte
 *                      aligned, scratch owned by the caller; without weights unused.
 * Repeated calls give the same bits. */
int fa2_rotary_bwd(const void* dq, const void* dk, const void* q, const void* k, const double* freqs,
                   const int* positions, const void* q_weight, const void* k_weight, void* q_grad, void* k_grad,
                   void* q_weight_grad, void* k_weight_grad, const long long* strides, int B, int Hq, int Hk, int N,
                   int d, int rotary_dim, int position_mode, int interleaved, float eps, float amplitude, int dtype,
                   int weight_dtype, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace of fa2_rotary_bwd; norm: with weights. 0 for invalid sizes. */
size_t fa2_rotary_bwd_workspace_size(int B, int Hq, int Hk, int N, int d, int norm);

/* Synchronises `stream`, then returns and clears the current device's status
 * word: FA2_OK, or FA2_ERR_DEVICE_TIMEOUT if any kernel since the last call
 * gave up on a bounded wait, else FA2_ERR_PAGE if a paged-cache kernel met a bad
 * page, length or count; or FA2_ERR_CUDA if the synchronisation failed. */
int fa2_get_device_status(void* stream);

/* Static, human-readable name of a status code. */
const char* fa2_status_string(int status);

/* ---- Host-only queries of the work mapping (no GPU needed) ----------------
 * Forward row blocks ("thread blocks" of "FlashAttention学习笔记(2)",
 * V2中的thread blocks排布) form the grid (num_m_block, B, H), the row block
 * varying fastest. Each owns rows_per_cta = 256 query rows (two 128-row
 * tiles). The split forward launches one CTA per (row block, part); the
 * unsplit one runs the row blocks on a persistent grid (fa2_fwd_schedule). */
int fa2_fwd_grid(int B, int H, int N, int grid_out[3], int* rows_per_cta);

/* Query rows [*row_begin, *row_end) and the number of K/V tiles of 128 keys
 * that forward row block `block_x` loads (causal: fully masked tiles are
 * skipped, "flash-attention123和ring-attention", 优化3). */
int fa2_fwd_block_work(int block_x, int N, int causal, int* row_begin, int* row_end,
                       int* kv_tiles);

/* Schedule of the unsplit forward on a device with num_sms multiprocessors:
 * *num_ctas CTAs (at most num_sms), each running a fixed list of row blocks.
 * Without a causal mask the row blocks are dealt round robin; with one, pairs
 * of row blocks q and num_m_block-1-q (a constant K/V total) are dealt round
 * robin, and the pairs left for a last partial round are the most balanced
 * ones of the last heads, run as halves. cta_of_block and pos_of_block (host
 * arrays of B*H*num_m_block ints, in fa2_fwd_grid order; either may be NULL)
 * receive each row block's CTA and its position in that CTA's list.
 * Returns FA2_ERR_INVALID_ARG for sizes < 1, causal not 0/1 or a NULL num_ctas. */
int fa2_fwd_schedule(int B, int H, int N, int causal, int num_sms, int* num_ctas, int* cta_of_block,
                     int* pos_of_block);

/* Backward dK/dV work = (num_n_block, B, H): one worker per 128-key column
 * block ("FlashAttention学习笔记(2)", Foward和backward中的thread block划分). The
 * main launch runs these workers, then the dQ workers, on a persistent grid
 * of at most one CTA per SM. */
int fa2_bwd_grid(int B, int H, int N, int d, int grid_out[3], int* keys_per_cta,
                 int* q_rows_per_tile);

/* Keys [*key_begin, *key_end) of backward column block `block_x` and the query
 * tiles [*q_tile_begin, *q_tile_end) (of q_rows_per_tile rows) it visits. */
int fa2_bwd_block_work(int block_x, int N, int d, int causal, int* key_begin, int* key_end,
                       int* q_tile_begin, int* q_tile_end);

/* ---- Diagnostics ----------------------------------------------------------
 * fa2_fwd, plus: tile_counts (device int array with one slot per forward row block,
 * grid order x fastest, or NULL) receives the number of K/V tiles loaded for
 * each row block. */
int fa2_fwd_instrumented(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                         int H, int N, int d, int causal, float scale, int dtype, int* tile_counts,
                         void* stream);

/* The CUDA runtime error code (cudaError_t; a driver CUresult plus 1000 for a
 * failed tensor-map encode) behind the last FA2_ERR_CUDA this thread received,
 * or 0. */
int fa2_last_cuda_error(void);

/* Arms a host-side fault for the next call of its kind in this process. Each
 * kind makes one TMA producer warp skip one load, so that a consumer's bounded
 * wait on it runs out after timeout_ms (1..5000) milliseconds instead of the
 * default 2 s; the kernel then records FA2_ERR_DEVICE_TIMEOUT, lets the copies
 * and MMAs it issued finish, frees its tensor memory and returns:
 *   1  the next fa2_fwd / fa2_fwd_qk / fa2_fwd_instrumented: the first V tile;
 *   2  the next fa2_fwd_split: the first V tile of every part;
 *   3  the next backward (fa2_bwd, fa2_bwd_atomic and their variants): the
 *      first dO tile of every K/V column worker;
 *   4  the next fa2_bwd (or fa2_bwd_qk, fa2_bwd_noalloc): the first V tile of
 *      every dQ worker;
 *   6  the next fa2_key_weights: the first Q tile of every CTA (there is no 5);
 *   7  the next fa2_prefix_decode whose prefix has a kernel of its own (any of more
 *      than 128 query rows to a key head): the first V tile of each of its CTAs;
 *   0  disarms.
 * Outputs of the faulted call are undefined. Exists to test the failure path
 * without hanging or faulting the GPU. */
int fa2_debug_arm_fault(int kind, int timeout_ms);

#ifdef __cplusplus
}
#endif

#endif /* FA2_H_ */
