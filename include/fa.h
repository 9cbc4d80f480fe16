/*
 * fa.h — fused exact-attention forward pass on GB300 (sm_103a), C ABI.
 *
 * The operation ("CUDA Flash Attention: Online Softmax with Shared Memory
 * Tiling", Problem Statement; "FlashAttention dissected", section "Algorithmic
 * core in pseudocode"): for every batch b, head h and query row i,
 *
 *     O[b,h,i,:] = sum_j softmax_j(scale * q_i . k_j) * v_j
 *     lse[b,h,i] = log( sum_j exp(scale * q_i . k_j) )          (natural log)
 *
 * computed by one fused kernel that keeps a query tile on chip, sweeps the
 * key/value sequence tile by tile with the online-softmax update (running
 * maximum m, running denominator l, accumulator rescaled by exp(m_old - m_new);
 * "How Did I Write My First FlashAttention Kernel in CUDA?", pseudo-algorithm
 * steps 1-5) and never writes the N x N score matrix to memory.
 *
 * Every entry point is callable from C.  No torch type appears here.
 */
#ifndef FA_GB300_H
#define FA_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes of every entry point. */
typedef enum {
    FA_OK = 0,
    FA_ERR_INVALID_ARG = 1,  /* NULL pointer, size < 1, overflow, non-finite scale */
    FA_ERR_UNSUPPORTED = 2,  /* head dimension / dtype combination not built, size beyond TMA limits */
    FA_ERR_ALIGNMENT = 3,    /* a tensor base address is not 16-byte aligned */
    FA_ERR_CUDA = 4,         /* a CUDA runtime or driver call failed (see fa_last_error_message) */
    FA_ERR_TIMEOUT = 5,      /* a kernel gave up waiting on an internal barrier (device status) */
    FA_ERR_CAPACITY = 6,     /* rows appended to a full cache were dropped (device status) */
    FA_ERR_RANGE = 7         /* a page number or a position outside its range (device status) */
} fa_status_t;

/* Element type of q, k, v and o (the low 8 bits of every `dtype` argument). */
typedef enum {
    FA_DTYPE_F32 = 0,   /* fp32 in/out; the two contractions run on TF32 tensor cores */
    FA_DTYPE_BF16 = 1,  /* bf16 in/out; fp32 accumulation and softmax */
    FA_DTYPE_F16 = 2    /* fp16 in/out; fp32 accumulation and softmax */
} fa_dtype_t;

/*
 * Flags OR-ed into a `dtype` argument.
 *
 * FA_FLAG_CAUSAL: autoregressive attention, query i sees only the keys
 * j <= i + (N_kv - N_q) (N_q = N_kv: the usual lower-triangular mask; the
 * last query always sees every key, as a decode step against a key cache
 * does).  A query that sees no key (N_q > N_kv) gets O = 0 and lse = -inf.
 * Causal masking is not on the pages; this is the conventional reading.
 */
#define FA_FLAG_CAUSAL 0x100

/*
 * fa_fwd — enqueue the attention forward pass on `stream`.
 *
 *   q, k, v : device pointers, contiguous row-major [B, H, N, d] of `dtype`
 *             (read only; they may alias one another).
 *   o       : device pointer, [B, H, N, d] of `dtype`, written in full.
 *   lse     : device pointer, fp32 [B, H, N], natural-log units; may be NULL,
 *             which skips the store.
 *   B, H, N : batch, heads, sequence length (queries = keys = N), each >= 1.
 *   d       : head dimension: 64 or 128 for bf16 and fp16, 64 for fp32.
 *   scale   : finite score scale (1/sqrt(d) for the pages' attention).
 *   dtype   : an fa_dtype_t value, optionally OR FA_FLAG_CAUSAL.
 *   stream  : a cudaStream_t (NULL = the legacy default stream) on the
 *             current device; all pointers must be on that device.
 *
 * Ownership: the caller owns every buffer; the library allocates and frees
 * nothing on the device.  o and lse must not overlap the inputs or each other.
 *
 * Work distribution (no workspace is needed): one CTA per 256 query rows of
 * one (b, h).  When those CTAs underfill the GPU (fewer than one per SM),
 * or the last of several waves is at most half full (16-bit inputs, no
 * causal mask, N >= 4096), the affected query blocks split their keys into
 * 2 to 8 partitions that run as one thread-block cluster and combine their
 * partial results in distributed shared memory with the online-softmax
 * rescaling ("FlashAttention dissected", sections "The mathematical
 * breakthrough: Tiling and Online Softmax" and "Interaction with the KV
 * cache during inference"); see fa_fwd_launches.  This is fa_fwd_ex's
 * automatic plan (num_splits = 0) restricted to merges inside a cluster.
 *
 * Errors: argument checks run on the host before any CUDA call and return
 * FA_ERR_INVALID_ARG / FA_ERR_UNSUPPORTED / FA_ERR_ALIGNMENT without side
 * effects.  A failed launch returns FA_ERR_CUDA.  The call is asynchronous:
 * FA_OK means the kernels were enqueued; a kernel that aborted on a barrier
 * timeout is reported by fa_device_status().  There is no CPU fallback.
 */
int fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
           int64_t B, int64_t H, int64_t N, int64_t d, float scale, int dtype,
           void* stream);

/*
 * Kernel launches fa_fwd enqueues for these sizes on the current device: 1,
 * or 2 when the last wave's query blocks run split in a second launch; 0 for
 * invalid sizes.  The SM count and cluster occupancy of the current device
 * are the CUDA queries here (without a device the plan is one launch).
 */
int fa_fwd_launches(int64_t B, int64_t H, int64_t N, int64_t d, int dtype);

/*
 * fa_fwd_validate — the host-side argument checks of fa_fwd, alone.  Returns
 * the status fa_fwd would return before touching CUDA.  Makes no CUDA call,
 * so it also runs on machines without a GPU.
 */
int fa_fwd_validate(const void* q, const void* k, const void* v, void* o,
                    const float* lse, int64_t B, int64_t H, int64_t N,
                    int64_t d, float scale, int dtype);

/*
 * fa_fwd_ex — the general form: decode shapes, grouped-query heads and
 * key-range partitions ("split-KV").
 *
 *   q, o    : [B, H, N_q, d] of `dtype`;   k, v : [B, H_kv, N_kv, d];
 *   lse     : fp32 [B, H, N_q] or NULL.
 *   H_kv    : key/value heads, dividing H; query head h reads key/value
 *             head h / (H / H_kv) (grouped-query attention; H_kv = H is
 *             ordinary multi-head attention).
 *   N_q, N_kv: query rows and key/value rows per head (N_q = 1 is a decode
 *             step against a cache of N_kv keys, the FlashDecoding case of
 *             "FlashAttention dissected", section "Interaction with the KV
 *             cache during inference").
 *   num_splits: >= 1 key-range partitions per query block.  1 runs the fused
 *             kernel alone.  More partitions sweep disjoint key ranges in
 *             separate CTAs, which then fill the GPU when B * H * N_q is
 *             small; their partial results go to `workspace` and a second
 *             kernel merges them with the online-softmax rescaling.  The
 *             count is capped at 32 and at one partition per 128 keys.
 *             0 chooses automatically for the current device (one CTA per
 *             SM): a launch with fewer query blocks than SMs gets the
 *             fa_fwd_ex_splits count, merged inside thread-block clusters
 *             (distributed shared memory, no workspace, no merge kernel)
 *             when at most 8 partitions are wanted and every query block's
 *             cluster fits on the device at once, else through the
 *             workspace and the merge kernel; a launch of several waves
 *             whose last wave is at most half full (16-bit inputs,
 *             unmasked, query heads not packed, N_kv >= 4096) runs the full
 *             waves unsplit and the last wave's query blocks in a second
 *             launch, split along the keys (up to 4 partitions) into
 *             clusters that merge in-cluster; otherwise one partition.
 *   workspace, workspace_bytes: device scratch owned by the caller, 16-byte
 *             aligned, at least fa_fwd_ex_workspace_size(...) bytes; may be
 *             NULL when that size is 0.  Contents on entry do not matter.
 *
 * Same ownership, validation and error behaviour as fa_fwd; the workspace
 * must not overlap any tensor.  Every kernel of the call (one to three, see
 * fa_fwd_ex_launches) is enqueued on `stream`.
 */
int fa_fwd_ex(const void* q, const void* k, const void* v, void* o, float* lse,
              int64_t B, int64_t H, int64_t H_kv, int64_t N_q, int64_t N_kv,
              int64_t d, float scale, int dtype, int num_splits,
              void* workspace, size_t workspace_bytes, void* stream);

/* Host-side argument checks of fa_fwd_ex alone (no CUDA call, except the
 * SM-count query of the current device when num_splits = 0). */
int fa_fwd_ex_validate(const void* q, const void* k, const void* v, void* o,
                       const float* lse, int64_t B, int64_t H, int64_t H_kv,
                       int64_t N_q, int64_t N_kv, int64_t d, float scale,
                       int dtype, int num_splits, const void* workspace,
                       size_t workspace_bytes);

/*
 * Workspace bytes fa_fwd_ex needs for `num_splits` (after the same capping):
 * splits * B * H * N_q * (d + 4) * 4, or 0 when one partition remains.
 * Pure host computation; 0 for invalid sizes.  num_splits = 0 (automatic):
 * a bound for every plan on the current device, min(SMs * 256,
 * 32 * B * H * N_q) * (d + 4) * 4 (SMs taken as 1024 when no device answers;
 * the SM count is the one CUDA query here).
 */
size_t fa_fwd_ex_workspace_size(int64_t B, int64_t H, int64_t N_q, int64_t N_kv,
                                int64_t d, int num_splits);

/*
 * A partition count that fills about one wave of `num_sms` SMs: 1 when the
 * CTAs of one partition already fill the GPU, else num_sms / that count
 * (capped as above).  A partition has B * H * ceil(N_q / 256) CTAs, or
 * B * H_kv when the grouped query heads are packed (H_kv < H and
 * N_q * H / H_kv <= 128: one CTA serves all query heads of a key/value head,
 * e.g. for decode steps).  Pure host computation; 1 for invalid sizes.
 */
int fa_fwd_ex_splits(int64_t B, int64_t H, int64_t H_kv, int64_t N_q, int64_t N_kv,
                     int num_sms);

/*
 * Kernel launches fa_fwd_ex enqueues for these arguments: 1 (one key
 * partition, or partitions merged in-cluster), 2 (partitions and their
 * merge kernel, or num_splits = 0 with a split tail: the full waves, then
 * the tail's clusters), 3 (partitions through the workspace, their merge and
 * a tail launch; not produced by the current plan); 0 for invalid sizes.  For num_splits = 0 the plan is the current device's (the
 * SM-count query is the one CUDA call here).
 */
int fa_fwd_ex_launches(int64_t B, int64_t H, int64_t H_kv, int64_t N_q, int64_t N_kv,
                       int64_t d, int dtype, int num_splits);

/*
 * fa_fwd_ex_static — fa_fwd_ex for callers that cannot allocate device
 * memory (plugins of engines that own the whole device memory pool, or
 * per-step code that must not call cudaMalloc, which can synchronise the
 * device and can fail at run time).  Same arguments and results as
 * fa_fwd_ex without the workspace: the split partials go to one static
 * device array of fa_fwd_ex_static_capacity() bytes (32 MiB) that the library
 * holds on every GPU that loads it, until the process exits.  The library
 * allocates nothing.
 *
 *   - Sizes whose partials exceed the capacity return FA_ERR_UNSUPPORTED
 *     (fa_fwd_ex_workspace_size() gives the bytes a call needs).
 *   - The first call on a device (and the first after a device reset)
 *     looks up the array's device address (cudaGetSymbolAddress) with that
 *     device current; make that first call before any stream capture.
 *   - Plans that merge their partitions inside thread-block clusters (see
 *     fa_fwd_ex, num_splits = 0) do not touch the array.
 *   - Every call on a device shares the array, which keeps the last call's
 *     contents (nothing in it needs to start at zero).  Calls whose kernels
 *     may overlap on the GPU race on it: serialise them.
 *
 * The pages have no counterpart of this entry point.
 */
int fa_fwd_ex_static(const void* q, const void* k, const void* v, void* o,
                     float* lse, int64_t B, int64_t H, int64_t H_kv,
                     int64_t N_q, int64_t N_kv, int64_t d, float scale,
                     int dtype, int num_splits, void* stream);

/* Bytes of the static array fa_fwd_ex_static uses, per device. */
size_t fa_fwd_ex_static_capacity(void);

/*
 * fa_fwd_host — fa_fwd_ex on tensors in HOST memory: the inputs are copied
 * to the GPU, the forward pass runs, and o and lse are copied back, with the
 * copies of one chunk of key/value heads overlapped with the computation of
 * the previous one (three streams: the caller's `stream` for the kernels and
 * two the library creates once per device).  Same arguments, layouts, dtypes,
 * flags and checks as fa_fwd_ex with num_splits = 1, except:
 *   q, k, v, o, lse : host memory; pinned (page-locked) memory is needed
 *                     for the copies to overlap (pageable memory works but
 *                     serialises them).
 *   workspace       : caller-owned DEVICE memory of at least
 *                     fa_fwd_host_workspace_size(...) bytes, 256-byte
 *                     aligned (three chunk slots of q, k, v, o, lse).
 * Completion: when `stream` reaches the point after this call, o and lse
 * hold the results in host memory.  Calls on one device share the two
 * internal streams (a mutex serialises their enqueueing).  Returns as
 * fa_fwd_ex; FA_ERR_INVALID_ARG for a missing or short workspace,
 * FA_ERR_ALIGNMENT for a workspace not 256-byte aligned.
 * The pages have no counterpart of this entry point; it is the host-to-host
 * form of the forward pass that end-to-end measurements call.
 */
int fa_fwd_host(const void* q, const void* k, const void* v, void* o, float* lse,
                int64_t B, int64_t H, int64_t H_kv, int64_t N_q, int64_t N_kv,
                int64_t d, float scale, int dtype, void* workspace,
                size_t workspace_bytes, void* stream);

/* Device workspace bytes fa_fwd_host needs (0 for invalid sizes). */
size_t fa_fwd_host_workspace_size(int64_t B, int64_t H, int64_t H_kv, int64_t N_q,
                                  int64_t N_kv, int64_t d, int dtype);

/*
 * fa_bwd — gradients of exact attention for an upstream gradient dO:
 *
 *   P = softmax(scale Q K^T) (recomputed from q, k and the saved lse),
 *   dV = P^T dO,  dS = P o (dO V^T - D),  D_i = dO_i . O_i,
 *   dQ = scale dS K,  dK = scale dS^T Q.
 *
 * "FlashAttention dissected", section "Memory complexity: from O(N^2) to
 * O(N)": the backward pass recomputes the attention blocks from Q, K, V and
 * the saved softmax statistics instead of storing the N x N matrix; the
 * gradient is the exact one of the forward definition (the pages give no
 * formula; this is the chain rule through O = P V and the softmax formula of
 * the same page).  The causal mask and grouped heads are those of fa_fwd_ex.
 *
 * Layout (contiguous, row-major, dtype = the inputs' dtype):
 *   q, o, dout, dq : [B, H, N_q, d]      k, v, dk, dv : [B, H_kv, N_kv, d]
 *   lse            : fp32 [B, H, N_q], natural log, as fa_fwd / fa_fwd_ex
 *                    return it (a row with no visible key: -inf)
 *   o and lse must be the forward outputs for the same q, k, v, scale and
 *   mask; dk and dv sum over the H / H_kv query heads sharing a key/value
 *   head.
 * dtype: FA_DTYPE_BF16 or FA_DTYPE_F16, optionally | FA_FLAG_CAUSAL;
 *   FA_DTYPE_F32 returns FA_ERR_UNSUPPORTED.  d: 64 or 128.
 * workspace: caller-owned device memory of at least
 *   fa_bwd_workspace_size(B, H, N_q, d) bytes, 16-byte aligned (fp32 row
 *   statistics and the fp32 dQ accumulator; nothing needs to be zeroed).
 * Ownership and errors: as fa_fwd_ex.  Every pointer must be non-NULL and
 *   16-byte aligned (lse 4-byte); dq, dk, dv and the workspace must not
 *   overlap any input or one another (inputs may alias one another).
 *   Validation failures return before any CUDA call.  Three kernels are
 *   enqueued on `stream`; the call does not wait for them.
 */
int fa_bwd(const void* q, const void* k, const void* v, const void* o,
           const void* dout, const float* lse, void* dq, void* dk, void* dv,
           int64_t B, int64_t H, int64_t H_kv, int64_t N_q, int64_t N_kv,
           int64_t d, float scale, int dtype, void* workspace,
           size_t workspace_bytes, void* stream);

/* The argument checks of fa_bwd alone; never touches the GPU. */
int fa_bwd_validate(const void* q, const void* k, const void* v, const void* o,
                    const void* dout, const float* lse, void* dq, void* dk,
                    void* dv, int64_t B, int64_t H, int64_t H_kv, int64_t N_q,
                    int64_t N_kv, int64_t d, float scale, int dtype,
                    const void* workspace, size_t workspace_bytes);

/*
 * fa_bwd_host — fa_bwd on tensors in HOST memory (q, k, v, o, dout, lse in;
 * dq, dk, dv out), with the copies of one chunk of key/value heads
 * overlapped with the computation of the previous one, as fa_fwd_host does
 * (it shares that entry point's two internal streams).  Same arguments,
 * layouts, dtypes, flags and checks as fa_bwd, except: the tensors are host
 * memory (pinned for the copies to overlap), and `workspace` is device
 * memory of at least fa_bwd_host_workspace_size(...) bytes, 256-byte
 * aligned.  Completion on `stream` means dq, dk, dv are in host memory.
 * The pages have no counterpart of this entry point.
 */
int fa_bwd_host(const void* q, const void* k, const void* v, const void* o,
                const void* dout, const float* lse, void* dq, void* dk, void* dv,
                int64_t B, int64_t H, int64_t H_kv, int64_t N_q, int64_t N_kv,
                int64_t d, float scale, int dtype, void* workspace,
                size_t workspace_bytes, void* stream);

/* Device workspace bytes fa_bwd_host needs (0 for invalid sizes). */
size_t fa_bwd_host_workspace_size(int64_t B, int64_t H, int64_t H_kv, int64_t N_q,
                                  int64_t N_kv, int64_t d);

/* Workspace bytes fa_bwd needs (0 for invalid sizes):
   8 * B * H * ceil(N_q / 128) * 128 (rounded up to 256) + 4 * B * H * N_q * d. */
size_t fa_bwd_workspace_size(int64_t B, int64_t H, int64_t N_q, int64_t d);

/* ------------------------------------------------------------------------
 * The 4-bit key/value cache.
 *
 * Decode steps against a long cache are bound by reading it.  This cache
 * holds keys and values in 4 bits and a scale per 16 channels (4.5 bits a
 * value, 0.28 of a 16-bit cache).  fa_kv4_append stores rows, fa_kv4_read
 * returns them, fa_kv4_fwd attends over them, fa_fwd_weights and fa_kv4_fwd
 * accumulate the attention weight each entry receives, and fa_kv4_evict keeps
 * the entries with the largest weight.  The pages have no counterpart of
 * these entry points; the attention is the pages' (online softmax over key
 * partitions, "FlashAttention dissected", sections "Algorithmic core in
 * pseudocode" and "Interaction with the KV cache during inference").
 *
 * Format.  A row (one token of one key/value head) is cut into blocks of 16
 * consecutive channels.  Per block
 *     s = e4m3(max |x| / 6)       nearest, ties to even, at most 448
 *     c = e2m1(x / s)             nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with
 *                                 its sign, ties to the even code, at most 6
 * and the stored value is c * s, which has at most 6 significant bits and
 * lies in 2^-10 .. 2688: bf16 and fp16 both hold it exactly, and nothing
 * below rounds it again.  s = 0: the block holds zeros (the sign of a zero is
 * not defined).  A block with an infinity or a NaN gets the scale NaN and
 * reads as NaN throughout.  There is no scale per head or tensor beside the
 * blocks': a block whose largest magnitude is at most 6 * 2^-10 (0.0059) is
 * stored as zeros, one below 6 * 2^-6 (0.094) has a scale of fewer bits, one
 * above 2688 saturates, all without a report.  Keys or values outside that
 * range are multiplied by a power of two before they are stored, and `scale`
 * (keys) or the output (values) by its inverse.  Two codes share a byte, the even channel in the
 * low half.
 *
 * Entries are slots 0 .. length - 1 of each key/value head; attention does
 * not depend on their order.  The library never allocates: every array is
 * the caller's, on the current device.
 */
typedef struct {
    uint8_t* k_codes;   /* [B, H_kv, capacity, d / 2], 16-byte aligned */
    uint8_t* k_scales;  /* [B, H_kv, capacity, d / 16] e4m3, 16-byte aligned */
    uint8_t* v_codes;   /* as k_codes */
    uint8_t* v_scales;  /* as k_scales */
    float* weight;      /* [B, H_kv, capacity] accumulated attention weight, or NULL */
    int32_t* pos;       /* [B, H_kv, capacity] position of the token in its sequence, or NULL */
    int32_t* counts;    /* [2, B]: slots in use (the length), then tokens appended so far */
    int64_t B, H_kv;
    int64_t capacity;   /* slots per key/value head, a multiple of 128 */
    int64_t d;          /* 64 or 128 */
} fa_kv4_cache_t;

/*
 * fa_kv4_append — store n rows per sequence at slots length .. length + n - 1.
 *
 *   k, v       : [B, H_kv, n, d] bf16 or fp16 (`dtype`, no flags), contiguous,
 *                16-byte aligned.
 *   counts_out : int32 [2, B], receives length + n and appended + n; may be
 *                the cache's own counts (advanced in place), which are left
 *                alone otherwise.
 * pos, where the cache has it, gets appended + i for row i, and weight 0.
 * Rows that do not fit the capacity are dropped, the length stops at the
 * capacity, and fa_device_status reports FA_ERR_CAPACITY.  One kernel, and a
 * second when counts advance in place and more than 1024 blocks of 16
 * channels are stored.
 */
int fa_kv4_append(const fa_kv4_cache_t* cache, const void* k, const void* v, int64_t n, int dtype,
                  int32_t* counts_out, void* stream);

/*
 * fa_kv4_read — the stored values of `count` slots of every head as bf16 or
 * fp16 rows k, v [B, H_kv, count, d] (exact; see the format), from slot
 * first[b] on (int32 [B] on the device; NULL: from slot 0).  Slots outside
 * 0 .. capacity - 1 read as zero; slots at or behind the length hold what was
 * there.  k or v may be NULL.  With it a chunk of a long prompt attends over
 * stored rows by fa_fwd_ex.
 */
int fa_kv4_read(const fa_kv4_cache_t* cache, const int32_t* first, int64_t count, void* k, void* v,
                int dtype, void* stream);

/*
 * fa_kv4_fwd — attention of q [B, H, N_q, d] over the cache's entries:
 *
 *     O = softmax(scale q K^T) V,  lse = log sum exp(scale q K^T)
 *
 * over the first counts[b] slots of key/value head h / (H / H_kv).
 *   o          : [B, H, N_q, d] of `dtype`;  lse: fp32 [B, H, N_q] or NULL.
 *   weight_out : fp32 [B, H_kv, capacity] or NULL.  Entry j of a head gets
 *                cache.weight (0 where that is NULL) plus the softmax weights
 *                of slot j, summed over the head's H / H_kv query heads and
 *                N_q rows; may be cache.weight itself.  Slots at or behind
 *                the length are not written.
 *   dtype      : FA_DTYPE_BF16 or FA_DTYPE_F16, optionally FA_FLAG_CAUSAL:
 *                row i sees slots j < length - (N_q - 1 - i), as the last N_q
 *                tokens do that were appended before the call.
 *   N_q * H / H_kv <= 128 (decode steps and drafts; longer chunks read the
 *   rows back with fa_kv4_read and use fa_fwd_ex): else FA_ERR_UNSUPPORTED.
 *   workspace  : fa_kv4_fwd_workspace_size(...) bytes, 16-byte aligned;
 *                nothing in it needs to be zeroed.  Calls (and replays of
 *                captured ones) that may run at once need one each.
 * A row that sees no slot gets O = 0 and lse = -inf and adds no weight.
 * Scores, sums, lse and the accumulated weights are held in 32 bits.  For the
 * product with V the softmax weights are rounded to fp16, to 2^-11 of each and
 * 2^-32 of the largest, and divided by the sum of the rounded ones.
 * Lengths are read on the device (clamped to 0 .. capacity), so a captured
 * call follows them.  Results do not depend on the order in which blocks run.
 * One or two kernels.
 */
int fa_kv4_fwd(const fa_kv4_cache_t* cache, const void* q, void* o, float* lse, float* weight_out,
               int64_t H, int64_t N_q, float scale, int dtype, void* workspace, size_t workspace_bytes,
               void* stream);

/* Workspace bytes of fa_kv4_fwd on the current device (the SM count is the
 * one CUDA query; 1024 SMs when no device answers); 0 for invalid sizes. */
size_t fa_kv4_fwd_workspace_size(int64_t B, int64_t H, int64_t H_kv, int64_t N_q, int64_t capacity, int64_t d,
                                 int with_weight);

/*
 * fa_kv4_evict — keep the `keep` entries of each key/value head that carry
 * the largest weight.
 *
 *   rank_by    : fp32 [B, H_kv, capacity], the weights to go by; NULL:
 *                cache.weight.  A NaN counts as larger than any number.
 *   sinks, recent : entries with pos < sinks or pos >= appended - recent are
 *                kept before all others (pos is needed when either is > 0).
 *                Ties, and any two of those, go to the lowest slot.
 *   to         : NULL: in place.  Else a cache of the same B, H_kv and d with
 *                capacity >= keep, sharing no memory with the first, which
 *                gets the kept entries and leaves the first as it was.  It
 *                gets pos and weight where both caches have them.
 *   src        : int32 [B, H_kv, keep]: the slot each slot's entry came from,
 *                -1 behind the last.
 *   counts_out : int32 [2, B]: min(length, keep) and appended; may be either
 *                cache's counts, which are left alone otherwise.
 * Slot j < min(length, keep) keeps its entry where that is kept; the other
 * slots there take, in order, the kept entries from behind them.  Slots at or
 * behind the new length are left as they were.  keep >= 1; capacity up to
 * 393216.  One kernel, another for copies into `to` and one to advance the
 * first cache's own counts.
 */
int fa_kv4_evict(const fa_kv4_cache_t* cache, int64_t keep, int64_t sinks, int64_t recent,
                 const float* rank_by, const fa_kv4_cache_t* to, int32_t* src, int32_t* counts_out,
                 void* stream);

/*
 * fa_fwd_weights — the attention weight that the keys of a prompt receive:
 *
 *     out[b, g, j] = in[b, g, j] + sum over the query heads h of group g and
 *                    rows i >= first_query of exp(scale q_i . k_j - lse_i)
 *
 * where row i sees key j.  q [B, H, N_q, d] and k [B, H_kv, N_kv, d] bf16 or
 * fp16, lse as fa_fwd / fa_fwd_ex returned it for the same scale and mask
 * (dtype's FA_FLAG_CAUSAL); rows whose lse is -inf count nothing.
 *   weight_in  : fp32, rows of N_kv values `weight_stride` apart (>= N_kv; a
 *                cache's weight has stride capacity), or NULL for zeros.
 *   weight_out : the same layout; may be weight_in.
 * Each output is summed by one thread in a fixed order: results repeat bit
 * for bit.  One kernel; no workspace.
 */
int fa_fwd_weights(const void* q, const void* k, const float* lse, const float* weight_in, float* weight_out,
                   int64_t weight_stride, int64_t B, int64_t H, int64_t H_kv, int64_t N_q, int64_t N_kv,
                   int64_t d, int64_t first_query, float scale, int dtype, void* stream);

/* The host-side argument checks of the calls above, alone; no CUDA call but
 * fa_kv4_fwd_workspace_size's query. */
int fa_kv4_append_validate(const fa_kv4_cache_t* cache, const void* k, const void* v, int64_t n, int dtype,
                           const int32_t* counts_out);
int fa_kv4_read_validate(const fa_kv4_cache_t* cache, const int32_t* first, int64_t count, const void* k,
                         const void* v, int dtype);
int fa_kv4_fwd_validate(const fa_kv4_cache_t* cache, const void* q, const void* o, const float* lse,
                        const float* weight_out, int64_t H, int64_t N_q, float scale, int dtype,
                        const void* workspace, size_t workspace_bytes);
int fa_kv4_evict_validate(const fa_kv4_cache_t* cache, int64_t keep, int64_t sinks, int64_t recent,
                          const float* rank_by, const fa_kv4_cache_t* to, const int32_t* src,
                          const int32_t* counts_out);
int fa_fwd_weights_validate(const void* q, const void* k, const float* lse, const float* weight_in,
                            const float* weight_out, int64_t weight_stride, int64_t B, int64_t H, int64_t H_kv,
                            int64_t N_q, int64_t N_kv, int64_t d, int64_t first_query, float scale, int dtype);

/* ------------------------------------------------------------------------
 * Attention over packed sequences.
 *
 * A batch of sequences of different lengths, their rows one behind the other
 * without padding: sequence s has query rows cu_q[s] .. cu_q[s + 1] - 1 of a
 * [T_q, H, d] tensor and key/value rows cu_k[s] .. cu_k[s + 1] - 1 of a
 * [T_k, H_kv, d] one.  The attention and its gradients are those of fa_fwd_ex
 * and fa_bwd within each sequence; the pages have no counterpart of the layout.
 *
 * A view of such a tensor: rows and heads may lie apart (q, k and v as slices
 * of one projection's output), the d elements of a row are contiguous.
 */
typedef struct {
    void* data;          /* row 0 of head 0, 16-byte aligned (NULL only where the view has no rows) */
    int64_t row_stride;  /* elements from a row to the next one of its head, a multiple of 8 */
    int64_t head_stride; /* elements from a head's row to the next head's, a multiple of 8 */
} fa_rows_t;

/*
 * fa_packed_fwd — O = softmax(scale Q K^T) V and lse, sequence by sequence.
 *
 *   q, o       : views of T_q rows and H heads;  k, v: of T_k rows and H_kv
 *                heads (H_kv divides H; query head h reads h / (H / H_kv)).
 *                No two rows of a view overlap: either all heads of a row come
 *                before the next row, or all rows of a head before the next.
 *   lse        : fp32 [H, T_q], natural log, or NULL.
 *   cu_q, cu_k : int32 [B + 1] on the device, read there: not decreasing, from 0
 *                or above up to T_q (T_k) or below; cu_k may be cu_q.  (Other
 *                values are clamped to that: no row outside the tensors is read
 *                or written, but what is computed is not defined.)
 *   B >= 1; T_q, T_k >= 0, T_q + 128 B and T_k + 128 B below 2^31.
 *   dtype      : FA_DTYPE_BF16 or FA_DTYPE_F16, optionally FA_FLAG_CAUSAL: of a
 *                sequence with n_q queries and n_k keys, query i sees keys
 *                j <= i + n_k - n_q.  d: 64 or 128.
 * A query that sees no key gets O = 0 and lse = -inf.  Rows of o and lse that
 * belong to no sequence are left as they were, and whatever the rows of other
 * sequences or of none hold (infinities, NaN) does not enter a sequence's
 * results.  Within a sequence, an infinity or a NaN in a value row may reach
 * queries that do not see it, as masked keys are multiplied with weight 0: those
 * whose last visible key is fewer than 128 rows before it, where H / H_kv is odd
 * fewer than 256, and 127 more where n_k - n_q is no multiple of 128 (keys go by
 * whole tiles of 128, up to the last that a block of 128 or 256 queries sees).
 * o overlaps no input.
 * Scores, sums and lse are held in 32 bits; the weights are rounded to `dtype` for
 * their product with V and divided by their sum, in which each tile's largest one is
 * the rounded one.  The product's sum over a sequence's n keys is one fp32 sum on the
 * tensor cores, which cut off what lies below its last bits: it is off by up to
 * n 2^-27 of the sum of |P| |V| (2^20 keys of like weight, values of one sign: 0.6 %,
 * 2^18: 0.12 %).
 * Results do not depend on the order in which blocks run.  One kernel; no workspace.
 */
int fa_packed_fwd(const fa_rows_t* q, const fa_rows_t* k, const fa_rows_t* v, const fa_rows_t* o, float* lse,
                  const int32_t* cu_q, const int32_t* cu_k, int64_t B, int64_t T_q, int64_t T_k, int64_t H,
                  int64_t H_kv, int64_t d, float scale, int dtype, void* stream);

/*
 * fa_packed_bwd — gradients of fa_packed_fwd: views dq of T_q rows and H heads,
 * dk and dv of T_k rows and H_kv heads, from the forward's o and lse and the
 * upstream gradient dout.  Arguments as in fa_packed_fwd; dk and dv sum over the
 * query heads that share a key/value head.
 *   workspace : fa_packed_bwd_workspace_size(...) bytes, 16-byte aligned;
 *               nothing in it needs to be zeroed.  Calls (and replays of
 *               captured ones) that may run at once need one each.  Its size,
 *               H (T_q / 128 + B) (512 d + 1024) + 128 bytes, grows with the
 *               sequences beside the rows: an fp32 row of dQ for each query row,
 *               and up to 127 more for each sequence (24000 rows of 16 heads, d = 128,
 *               in 8 sequences 0.21 GB, in 1000 1.26, in 4000 4.46).
 * Rows of dq, dk and dv that belong to no sequence are left as they were; keys
 * that no query sees get zeros.  Non-finite rows of o, dout, q, k or v stay in
 * their sequence (in it they may reach gradients of rows that the mask hides from
 * them).  dq, dk, dv and the workspace overlap no input and
 * not each other (slices of one tensor are fine: of its heads, or parts beside each head).  dQ is summed over the key
 * blocks in fp32 in an order that may change from call to call, as in fa_bwd;
 * dk and dv repeat bit for bit.  P and dS are rounded to `dtype` for their products;
 * dk and dv are one fp32 sum each over the H / H_kv n_q rows that reach a key, cut off as
 * the forward's.  Three kernels.
 */
int fa_packed_bwd(const fa_rows_t* q, const fa_rows_t* k, const fa_rows_t* v, const fa_rows_t* o,
                  const fa_rows_t* dout, const float* lse, const fa_rows_t* dq, const fa_rows_t* dk,
                  const fa_rows_t* dv, const int32_t* cu_q, const int32_t* cu_k, int64_t B, int64_t T_q,
                  int64_t T_k, int64_t H, int64_t H_kv, int64_t d, float scale, int dtype, void* workspace,
                  size_t workspace_bytes, void* stream);

/* Workspace bytes fa_packed_bwd needs (0 for invalid sizes). */
size_t fa_packed_bwd_workspace_size(int64_t B, int64_t T_q, int64_t H, int64_t d);

/* The host-side argument checks of the two calls, alone; no CUDA call. */
int fa_packed_fwd_validate(const fa_rows_t* q, const fa_rows_t* k, const fa_rows_t* v, const fa_rows_t* o,
                           const float* lse, const int32_t* cu_q, const int32_t* cu_k, int64_t B, int64_t T_q,
                           int64_t T_k, int64_t H, int64_t H_kv, int64_t d, float scale, int dtype);
int fa_packed_bwd_validate(const fa_rows_t* q, const fa_rows_t* k, const fa_rows_t* v, const fa_rows_t* o,
                           const fa_rows_t* dout, const float* lse, const fa_rows_t* dq, const fa_rows_t* dk,
                           const fa_rows_t* dv, const int32_t* cu_q, const int32_t* cu_k, int64_t B, int64_t T_q,
                           int64_t T_k, int64_t H, int64_t H_kv, int64_t d, float scale, int dtype,
                           const void* workspace, size_t workspace_bytes);

/* ------------------------------------------------------------------------
 * The paged 16-bit key/value cache.
 *
 * Keys and values of sequences of different lengths in pages of a common pool,
 * so that memory is handed out a page at a time and sequences may share pages
 * (a prompt's).  fa_paged_append rotates rows by their positions and stores
 * them, fa_paged_fwd attends over a sequence's pages, behind a prefix that all
 * sequences share, if there is one.  The attention is the pages' (online softmax
 * over key partitions, "FlashAttention dissected", sections "Algorithmic core in
 * pseudocode" and "Interaction with the KV cache during inference"); the layout
 * and the rotation have no counterpart there.
 *
 * Slot s of sequence b is row s % page_size of page block_table[b][s / page_size].
 * The library never allocates: every array is the caller's, on the current device.
 */
typedef struct {
    void* k_pages;              /* [num_pages, H_kv, page_size, d], 16-byte aligned, of the calls' dtype */
    void* v_pages;              /* as k_pages */
    const int32_t* block_table; /* [B, max_pages]; numbers behind a sequence's last slot are not looked at */
    int32_t* lengths;           /* [B]: slots in use, 0 .. max_pages * page_size (other values are clamped) */
    int64_t num_pages;
    int64_t page_size;          /* 16, 32, 64 or 128 */
    int64_t B, max_pages, H_kv;
    int64_t d;                  /* 64 or 128 */
} fa_paged_cache_t;

/* fa_paged_append: pairs of neighbouring channels are rotated (else channel j with j + rot / 2). */
#define FA_FLAG_INTERLEAVED 0x200

/*
 * fa_paged_append — store new rows of every sequence behind its last slot, keys
 * rotated by their positions, and rotate the queries beside them.
 *
 *   k, v       : views of T rows and H_kv heads;  cu: int32 [B + 1] on the
 *                device, rows cu[b] .. cu[b + 1] - 1 are sequence b's (not
 *                decreasing, within 0 .. T; with other values no row outside
 *                the tensors and the pool is read or written, but what is stored
 *                and the lengths are not defined), or NULL: T / B rows each.
 *   q, q_out   : views of T rows and H heads, or both NULL; q_out may be q.
 *   k_out      : view of T rows and H_kv heads that gets the rotated keys too
 *                (for fa_packed_fwd over a prompt), or NULL; may be k.
 *   table      : fp32 [table_rows, rot], 16-byte aligned: row p holds the cosines of
 *                position p's rot / 2 angles, then their sines; or NULL: nothing
 *                is rotated (q_out and k_out are copies).  rot: a multiple of 16 up to d, the
 *                channels that are rotated; the others are copied.
 *   positions  : int32 [T], the rows' positions, or NULL: first_position + the slot.
 *   lengths_out: int32 [B], receives the lengths with the new rows; may be the
 *                cache's own (advanced in place), which are left alone otherwise.
 *   dtype      : FA_DTYPE_BF16 or FA_DTYPE_F16, optionally FA_FLAG_INTERLEAVED.
 * Pair (x, y) becomes (x cos - y sin, x sin + y cos), in 32 bits, rounded once.
 * Key and value rows past max_pages * page_size slots are dropped and
 * fa_device_status reports FA_ERR_CAPACITY; those whose page number is outside the
 * pool are dropped, and positions outside the table are rotated as its first
 * or last row, and it reports FA_ERR_RANGE.  Rows of no sequence, and pages
 * but for the new rows, are left as they were.  Where two slots written are the
 * same row of the pool either may stay.  One kernel where lengths_out is not the
 * cache's, or where cu is NULL and each sequence has one row (in large batches, or of
 * few heads, a few); else, with cu or without rows too, a second one advances the lengths.
 */
int fa_paged_append(const fa_paged_cache_t* cache, const fa_rows_t* k, const fa_rows_t* v, const int32_t* cu,
                    int64_t T, const fa_rows_t* q, const fa_rows_t* q_out, int64_t H, const fa_rows_t* k_out,
                    const float* table, int64_t table_rows, int64_t rot, const int32_t* positions,
                    int64_t first_position, int32_t* lengths_out, int dtype, void* stream);

/*
 * fa_paged_fwd — attention of q [B, H, N_q, d] over the sequences' slots:
 *
 *     O = softmax(scale q K^T) V,  lse = log sum exp(scale q K^T)
 *
 * over key/value head h / (H / H_kv) of the prefix's prefix_length slots, which all
 * sequences share (read once for two tiles of up to 128 rows of whole sequences, so
 * for a batch of up to 256 rows a key/value head), followed by the sequence's own lengths[b].
 *   o            : [B, H, N_q, d] of `dtype`;  lse: fp32 [B, H, N_q] or NULL.
 *   prefix_pages : int32 [ceil(prefix_length / page_size)] on the device, pages of
 *                  the same pool; NULL exactly where prefix_length is 0.
 *   dtype        : FA_DTYPE_BF16 or FA_DTYPE_F16, optionally FA_FLAG_CAUSAL:
 *                  row i sees the prefix and the own slots
 *                  j < lengths[b] - (N_q - 1 - i).
 *   N_q * H / H_kv <= 128 (decode steps and drafts): else FA_ERR_UNSUPPORTED.  Above 32
 *                  the own slots' keys and values are read once for every 32.
 *   workspace    : fa_paged_fwd_workspace_size(...) bytes, 16-byte aligned;
 *                  nothing in it needs to be zeroed.  Calls (and replays of
 *                  captured ones) that may run at once need one each.
 * A row that sees no slot gets O = 0 and lse = -inf.  A page number outside the pool reads as
 * zeros.  What slots at or behind the length hold does not matter; an infinity
 * or a NaN in a value row that a draft's mask hides may reach that draft's rows.
 * Lengths, block table and prefix pages are read on the device, so a captured call
 * follows them.  Scores, sums and lse are held in 32 bits; the weights are rounded
 * to `dtype` for their product with V and divided by the sum of the rounded ones (the
 * prefix's, of its tiles' largest ones).  Results do not depend on the order
 * in which blocks run.  Two kernels, three with a prefix.
 */
int fa_paged_fwd(const fa_paged_cache_t* cache, const void* q, void* o, float* lse, int64_t H, int64_t N_q,
                 const int32_t* prefix_pages, int64_t prefix_length, float scale, int dtype, void* workspace,
                 size_t workspace_bytes, void* stream);

/* Workspace bytes of fa_paged_fwd on the current device, for a cache of B
 * sequences of up to `capacity` (max_pages * page_size) slots (the SM count is
 * the one CUDA query; 1024 SMs when no device answers); 0 for invalid sizes. */
size_t fa_paged_fwd_workspace_size(int64_t B, int64_t H, int64_t H_kv, int64_t N_q, int64_t capacity, int64_t d,
                                   int64_t prefix_length);

/* The host-side argument checks of the two calls, alone; no CUDA call but
 * fa_paged_fwd_workspace_size's query. */
int fa_paged_append_validate(const fa_paged_cache_t* cache, const fa_rows_t* k, const fa_rows_t* v, const int32_t* cu,
                             int64_t T, const fa_rows_t* q, const fa_rows_t* q_out, int64_t H,
                             const fa_rows_t* k_out, const float* table, int64_t table_rows, int64_t rot,
                             const int32_t* positions, int64_t first_position, const int32_t* lengths_out, int dtype);
int fa_paged_fwd_validate(const fa_paged_cache_t* cache, const void* q, const void* o, const float* lse, int64_t H,
                          int64_t N_q, const int32_t* prefix_pages, int64_t prefix_length, float scale, int dtype,
                          const void* workspace, size_t workspace_bytes);

/*
 * fa_device_status — synchronise `stream`, then read and clear the device
 * error word the kernels set when a bounded wait gives up, a cache overflows or
 * a number is out of its range.  Returns FA_OK, FA_ERR_TIMEOUT, FA_ERR_CAPACITY,
 * FA_ERR_RANGE (in this order, where several are set), or FA_ERR_CUDA
 * if the synchronisation itself failed.
 * A launch that timed out leaves its outputs incomplete (the CTAs of that
 * launch stop early); later launches run normally whether or not the word
 * has been read.
 *
 * Source: "CUDA Flash Attention: Online Softmax with Shared Memory Tiling",
 * Correctness Audit (13-Category Checklist), row "Async error surfacing"
 * (the fused kernel's launch errors are checked with cudaGetLastError).  The
 * page surfaces launch errors only; this call extends the same rule to
 * errors a kernel detects while it runs, which an asynchronous launch cannot
 * return.
 */
int fa_device_status(void* stream);

/*
 * fa_selftest_barrier_timeout — enqueue on `stream` a one-CTA kernel that
 * waits, with the forward kernel's bounded barrier wait (about 1 s), on a
 * barrier phase that nothing completes.  The wait gives up, the kernel exits
 * normally and fa_device_status(stream) then returns FA_ERR_TIMEOUT (once).
 * It exercises the failure-reporting path without faulting or hanging the
 * GPU; the context stays usable.  Returns FA_OK or FA_ERR_CUDA (launch).
 */
int fa_selftest_barrier_timeout(void* stream);

/*
 * Static English text for a status code; never NULL.
 *
 * Source: "CUDA Flash Attention: Online Softmax with Shared Memory Tiling",
 * Correctness Audit (13-Category Checklist), rows "Async error surfacing"
 * (cudaGetLastError after the launch) and "Latent coupling bugs" (the head
 * dimension is checked, assert(d==64), instead of assumed).  Here those
 * checks return status codes instead of aborting, and this call names them.
 */
const char* fa_status_string(int status);

/* Text of the last CUDA error seen by this thread's calls ("" if none). */
const char* fa_last_error_message(void);

/* Library version: major * 10000 + minor * 100 + patch. */
int fa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FA_GB300_H */
