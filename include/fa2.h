/*
 * fa2.h - C ABI of the GB300 (sm_103a) FlashAttention-2 forward library.
 *
 * The operation. Exact scaled-dot-product attention, forward pass only, as
 * defined for FlashAttention-2 in "A Case Study in CUDA Kernel Fusion:
 * Implementing FlashAttention-2 on NVIDIA Hopper Architecture using the
 * CUTLASS Library" (abstract: online softmax fused with two back-to-back
 * GEMMs), restricted to the slice listed under "Kernel Specification" in
 * "FlashAttention-2 from scratch on Ampere, Part 1" (lubitschian.com/flash/
 * Part-1): non-causal, equal query/key/value sequence lengths, sequence
 * lengths divisible by the block size, 16-bit (bf16 or fp16) inputs and
 * outputs, softmax in fp32. For every batch b, query head h and query row i:
 *
 *     S[j]   = scale * <Q[b,h,i,:], K[b,g(h),j,:]>        j = 0 .. N-1
 *     O[b,h,i,:] = sum_j softmax(S)[j] * V[b,g(h),j,:]
 *     LSE[b,h,i] = ln sum_j exp(S[j])                     (natural log)
 *
 * with g(h) = h / (Hq / Hkv). Grouped KV heads (Hq > Hkv) use the query-head
 * packing named in "FlashAttention-3 for Inference: INT8 Quantization and
 * Query Head Packing for MQA/GQA" (Colfax Research author page): the Hq/Hkv
 * query heads that share a KV head are consecutive, so their rows form one
 * contiguous block of Hq/Hkv * N query rows that is processed against a
 * single stream of K/V tiles. The N x N score matrix never reaches memory.
 *
 * Data layout. All tensors are dense, row-major, caller-owned device memory:
 *     q, o : [B, Hq,  N, d]   16-bit elements (bf16 or fp16, same for all)
 *     k, v : [B, Hkv, N, d]   16-bit elements
 *     lse  : [B, Hq,  N]      fp32
 * Every pointer must be 16-byte aligned. Outputs are fully overwritten.
 *
 * Execution. Calls are asynchronous on `stream` (0 = legacy default stream);
 * each forward call launches exactly one kernel, fa2_fwd_kv16 two and fa2_bwd
 * three (in stream order). The library allocates no memory per call;
 * it owns one status word per device (a __device__ variable), which the
 * kernel sets if one of its bounded waits gives up.
 *
 * Errors. Argument errors (FA2_ERR_INVALID_ARG) and unsupported sizes or
 * devices (FA2_ERR_UNSUPPORTED) are detected on the host before anything is
 * launched. FA2_ERR_CUDA means a CUDA call of the library failed; each launch
 * is judged by its own return code, so an error the caller left pending does
 * not turn a successful call into a failure, and a failed call leaves none
 * of its own (non-sticky) errors pending. No entry point exits the process
 * or throws.
 */
#ifndef FA2_H_
#define FA2_H_

#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FA2_BF16 = 0,
    FA2_FP16 = 1
} fa2_dtype;

typedef enum {
    FA2_OK = 0,
    FA2_ERR_INVALID_ARG = 1,  /* NULL/misaligned pointer, non-positive size,
                                 Hq % Hkv != 0, scale not finite and > 0 */
    FA2_ERR_UNSUPPORTED = 2,  /* d not in {64, 128}, N % 128 != 0, sizes past
                                 32-bit coordinates, or a device that is not
                                 compute capability 10.3 */
    FA2_ERR_CUDA = 3,         /* a CUDA runtime/driver call failed */
    FA2_ERR_TIMEOUT = 4,      /* the kernel's watchdog gave up on a wait */
    FA2_ERR_BOUNDS = 5        /* a device-side bounds check failed and the access
                                 was skipped: a page id, slot or length of the KV
                                 cache entry points, or anything in the debug
                                 build (libfa2_debug.so, compiled with FA2_DEBUG) */
} fa2_status;

/*
 * Multi-head attention forward (Hq == Hkv == H).
 *   q, k, v : [B, H, N, d] 16-bit, device, 16-byte aligned (inputs, read only)
 *   o       : [B, H, N, d] 16-bit, device (output)
 *   lse     : [B, H, N] fp32, device (output, natural-log logsumexp of the
 *             scaled scores)
 *   B, H, N : positive; N a multiple of 128
 *   d       : 64 or 128
 *   scale   : finite, > 0 (usually 1/sqrt(d))
 *   dtype   : element type of q, k, v and o
 *   stream  : CUDA stream the kernel is queued on
 * Returns FA2_OK once the kernel is queued; FA2_ERR_* otherwise, and then
 * nothing was launched.
 */
fa2_status fa2_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                   int B, int H, int N, int d, float scale, fa2_dtype dtype,
                   cudaStream_t stream);

/*
 * Grouped-KV (GQA/MQA) attention forward. Same contract as fa2_fwd, with
 * q, o : [B, H_q, N, d], k, v : [B, H_kv, N, d], lse : [B, H_q, N] and
 * H_q a multiple of H_kv; query head h reads KV head h / (H_q / H_kv).
 * fa2_fwd(..., H, ...) is fa2_fwd_gqa(..., H, H, ...).
 */
fa2_status fa2_fwd_gqa(const void* q, const void* k, const void* v, void* o, float* lse,
                       int B, int H_q, int H_kv, int N, int d, float scale,
                       fa2_dtype dtype, cudaStream_t stream);

/*
 * General attention forward: query and key lengths may differ and need not be
 * multiples of 128, with an optional causal mask. This goes beyond the
 * "Kernel Specification" of "FlashAttention-2 from scratch on Ampere,
 * Part 1" (equal lengths, non-causal, lengths divisible by the block size),
 * which excludes these variants; they are built here as extensions.
 *   q, o : [B, H_q, N_q, d]; k, v : [B, H_kv, N_k, d]; lse : [B, H_q, N_q]
 *   N_q, N_k : positive, any value
 *   causal   : 0 or 1. With 1, query row i attends key j iff
 *              j < min(N_k, i + 1 + N_k - N_q) (the mask aligned to the end of
 *              the key sequence; j <= i when N_q == N_k). A row with no
 *              allowed key gets O = 0 and LSE = -inf.
 * Other arguments, layouts and errors as fa2_fwd_gqa (causal not in {0, 1}
 * is FA2_ERR_INVALID_ARG; no N % 128 restriction). The non-causal
 * equal-length case with N % 128 == 0 runs the same kernel as fa2_fwd_gqa.
 */
fa2_status fa2_fwd_ex(const void* q, const void* k, const void* v, void* o, float* lse,
                      int B, int H_q, int H_kv, int N_q, int N_k, int d, float scale,
                      int causal, fa2_dtype dtype, cudaStream_t stream);

/*
 * FP8 attention forward with in-kernel scaling: the inference variant named
 * by "FlashAttention-3 for Inference: INT8 Quantization and Query Head
 * Packing for MQA/GQA" (Colfax Research author page: quantised inputs,
 * in-kernel pre-processing by specialised warps, query-head packing). The
 * pages give no more than that; the form here:
 *   q       : [B, H_q, N, d] e4m3 codes (OCP FP8 E4M3, one byte each), device
 *   k, v    : [B, H_kv, N, d] e4m3 codes, device
 *   q_descale, k_descale, v_descale : [B * H_kv] fp32, device; the value of
 *             a code of (batch b, KV head g) -- for q, of the query heads
 *             that share KV head g -- is code * descale[b * H_kv + g];
 *             each finite and >= 0 (negative descales: results undefined)
 *   o       : [B, H_q, N, d] bf16, device (output)
 *   lse     : [B, H_q, N] fp32, device (output, natural-log logsumexp of the
 *             scaled scores of the dequantised inputs)
 *   d       : 128 (other values: FA2_ERR_UNSUPPORTED)
 *   B, H_q, H_kv, N, scale, stream : as fa2_fwd_gqa (N % 128 == 0)
 * Both products run on e4m3 tensor-core operands: S = Q K^T exactly in fp32
 * (then scaled by scale * dq * dk), and the softmax weights are scaled by
 * 2^8 and rounded to e4m3 before P V; l sums the unrounded weights. So O
 * differs from attention on the dequantised inputs by at most
 * 2^-4 sum_j p_j |v_j| / l + 2^-18 sum_j |v_j| / l per element (plus the
 * bf16 rounding of O); the LSE carries no rounding of P.
 * Alignment: q, k, v, o, lse 16-byte aligned; descales 4-byte aligned.
 * Errors as fa2_fwd_gqa. Nothing is allocated; all buffers are the caller's.
 */
fa2_status fa2_fwd_fp8(const void* q, const void* k, const void* v, const float* q_descale,
                       const float* k_descale, const float* v_descale, void* o, float* lse,
                       int B, int H_q, int H_kv, int N, int d, float scale, cudaStream_t stream);

/*
 * fa2_fwd_fp8 generalised as fa2_fwd_ex generalises fa2_fwd_gqa: separate
 * query and key lengths, any N_q, N_k >= 1, and the optional bottom-right
 * causal mask (query row i attends keys j < min(N_k, i + 1 + N_k - N_q),
 * "FlashAttention-2 from scratch on Ampere, Part 1", Kernel Specification,
 * lists both as left out of its kernel; the reading is that of fa2_fwd_ex).
 *   q       : [B, H_q, N_q, d] e4m3 codes; o : [B, H_q, N_q, d] bf16;
 *   lse     : [B, H_q, N_q] fp32 (a row with no allowed key: o = 0,
 *             lse = -inf)
 *   k, v    : [B, H_kv, N_k, d] e4m3 codes
 *   descales, d, alignment, numerics: as fa2_fwd_fp8. Key tiles of 128
 *             start at key 0, so a masked row rounds its weights exactly as
 *             the unmasked method on its visible keys.
 *   causal  : 0 or 1 (other values FA2_ERR_INVALID_ARG)
 * Non-causal calls with N_q == N_k and N_q % 128 == 0 run fa2_fwd_fp8.
 * More than 2^31 - 1 query or key rows: FA2_ERR_UNSUPPORTED. Errors
 * otherwise as fa2_fwd_fp8. Nothing is allocated.
 */
fa2_status fa2_fwd_fp8_ex(const void* q, const void* k, const void* v, const float* q_descale,
                          const float* k_descale, const float* v_descale, void* o, float* lse,
                          int B, int H_q, int H_kv, int N_q, int N_k, int d, float scale, int causal,
                          cudaStream_t stream);

/*
 * Attention backward (gradients of the forward with optional causal mask and
 * equal query/key lengths N; any N >= 1, like fa2_fwd_ex). The forward pages exclude the
 * backward pass ("FlashAttention-2 from scratch on Ampere, Part 1", Kernel
 * Specification: forward pass only); it is built here as an extension and
 * recomputes P = exp(scale*S - LSE) from the forward's logsumexp:
 *     D = rowsum(dO o O), dP = dO V^T, dS = P o (dP - D),
 *     dQ = scale dS K, dK = scale dS^T Q, dV = P^T dO
 * (grouped KV heads: dK, dV summed over the query heads that share them).
 *   q, o, dout, dq : [B, H_q, N, d] 16-bit (q, o, dout read; dq written)
 *   k, v, dk, dv   : [B, H_kv, N, d] 16-bit (k, v read; dk, dv written)
 *   lse            : [B, H_q, N] fp32, the forward's logsumexp (read)
 *   delta          : [B, H_q, N] fp32, caller-owned workspace; the call
 *                    writes D into it and then reads it back
 *   causal         : 0 or 1 (same mask as the forward with N_q == N_k)
 * All pointers device memory, 16-byte aligned. Launches three kernels on
 * `stream` (D, then dK/dV, then dQ); allocates nothing. Errors as
 * fa2_fwd_gqa except that N need not be a multiple of 128; B*H_q > 65535
 * is FA2_ERR_UNSUPPORTED. If one of the three launches fails
 * (FA2_ERR_CUDA), the kernels before it may already be queued and the
 * gradients are undefined.
 */
fa2_status fa2_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse,
                   const void* dout, void* dq, void* dk, void* dv, float* delta,
                   int B, int H_q, int H_kv, int N, int d, float scale, int causal,
                   fa2_dtype dtype, cudaStream_t stream);

/*
 * fa2_bwd without the `delta` workspace, for callers that cannot allocate
 * device memory: a plugin handed only its input and output tensors by a host
 * framework that owns every device allocation, or code running where a
 * device allocation is not allowed or its implicit synchronisation cannot be
 * afforded. (The source pages have no counterpart; this is an interface
 * convenience of this library.)
 *
 * Same arguments and results as fa2_bwd minus `delta`. D = rowsum(dO o O)
 * lives instead in a fixed device array inside this library, sized for
 * B * H_q * N <= 1048576 query rows (4 MiB of fp32, held on every GPU that
 * loads the library until the process exits). Errors: first those of
 * fa2_bwd for the same arguments (so a NULL pointer is FA2_ERR_INVALID_ARG
 * whatever the size, and a device that is not compute capability 10.3 is
 * FA2_ERR_UNSUPPORTED), then more than 1048576 query rows is
 * FA2_ERR_UNSUPPORTED; nothing is launched in those cases. Nothing is
 * allocated by the call.
 * Each call looks up the array's device address in the current device's
 * context (cudaGetSymbolAddress, a host-side lookup), so the address stays
 * right after cudaDeviceReset or under another context. The first call on a
 * device may load this library's device code on it; make that first call
 * before any stream capture. Every call uses the same array: calls that may
 * overlap on the GPU (other streams, other host threads) race on it and
 * must be ordered by the caller. The array keeps the last call's D; each
 * call rewrites the rows it uses before reading them.
 */
fa2_status fa2_bwd_noalloc(const void* q, const void* k, const void* v, const void* o, const float* lse,
                           const void* dout, void* dq, void* dk, void* dv,
                           int B, int H_q, int H_kv, int N, int d, float scale, int causal,
                           fa2_dtype dtype, cudaStream_t stream);

/*
 * A paged KV cache held in 4 bits, for serving. (The source pages leave the
 * KV cache out; these four entry points extend the library.) The cache is the
 * caller's device memory, one block of bytes
 *     cache : [num_pages, H_kv, 2, page_size * (d/2 + d/16)]
 * Part 0 of a (page, KV head) holds the keys of page_size tokens, part 1 the
 * values: first the e2m1 codes [page_size, d/2] (OCP FP4 E2M1; element 2i of
 * a token in the low four bits of byte i), then an OCP FP8 E4M3 scale for each
 * 16 elements [page_size, d/16]. An element stands for
 *     code * scale * descale[h]
 * with k_descale, v_descale : [H_kv] fp32, device, finite and > 0 (a head's
 * largest magnitude over 6 * 448 uses the whole range). That is 4.5 bits an
 * element. A token's place is its slot, page * page_size + offset; request b's
 * position i lies in page block_table[b, i / page_size] at offset
 * i % page_size. Table entries behind a request's last page are never read.
 *   d         : 64 or 128
 *   page_size : 16, 32, 64 or 128; num_pages * page_size < 2^31 - 256
 *   block_table : [B, max_pages] int32, max_pages * page_size < 2^31 - 256
 * Page ids, slots and lengths come from device memory: one that points outside
 * the cache or the table is skipped on the device in every build and reported
 * by fa2_check_status as FA2_ERR_BOUNDS. Pointers: cache, tensors and
 * workspace 16-byte aligned, int32 and descale arrays 4-byte aligned. Errors
 * otherwise as fa2_fwd_gqa; nothing is allocated.
 */

/*
 * Pages and slots of one scheduling step, from the request lengths.
 *   seq_lens  : [B] int32, tokens that request b has in the cache
 *   new_lens  : [B] int32, tokens this step adds (0 .. N), or negative: the
 *               request ends and gives its pages back
 *   block_table : [B, max_pages] int32, in and out: the entries of new pages
 *               are written, all others stay as they were
 *   free_pages, free_state : a ring of free page ids [num_pages] int32 and
 *               {index of the first, how many} int32. New pages are taken from
 *               its front; pages given back are written behind its end and are
 *               handed out from the next call on
 *   seq_lens_out : [B] int32, the lengths after the step (may be seq_lens)
 *   accepted  : [B] int32, new_lens[b] if the request got its pages, else 0
 *   slots     : [B, N] int32, the slots of the accepted tokens, -1 in the
 *               other places
 *   free_state_out : [2] int32 (may be free_state)
 * Requests are served in order. One that needs pages gets them iff the pages
 * wanted by the requests up to and including it are free; one that needs none
 * (its last page has room) always gets its slots. new_lens[b] > N, or a length
 * that its table row cannot hold, is not accepted and wants no page. A length
 * below 0 or above max_pages * page_size counts as 0 and is reported, and so
 * is a ring that is not one. An id outside the cache in the row of a request that
 * ends is reported and does not join the ring; one in the ring itself is reported
 * when it is handed out, and the slots on it are -1. A page that two requests
 * share must be given back once only. B * N < 2^31 - 1024. One launch; calls that
 * share a ring must be ordered.
 */
fa2_status fa2_kv4_plan(const int32_t* seq_lens, const int32_t* new_lens, int32_t* block_table,
                        int32_t* free_pages, const int32_t* free_state, int32_t* seq_lens_out,
                        int32_t* accepted, int32_t* slots, int32_t* free_state_out, int B, int N,
                        int max_pages, int page_size, int num_pages, cudaStream_t stream);

/*
 * Quantises new keys and values and writes them into their slots.
 *   k, v   : [B, H_kv, N, d] bf16 or fp16, elements of a row adjacent; the
 *            strides of request, head and token are given in elements
 *            (multiples of 8, 0 .. 2^31 - 8) so that views of a
 *            projection's output need no copy
 *   slots  : [B, N] int32; a negative slot is skipped. A slot may be named
 *            once in a call: two tokens written to one slot at the same time
 *            leave codes of the one beside scales of the other
 * For each 16 elements x: scale = e4m3(max|x| / (6 descale)), t = scale *
 * descale in fp32, code = e2m1(x / t), every rounding to nearest, ties to
 * even, limited to the format's largest value; t = 0 gives codes 0. 16
 * elements that hold a NaN or an infinity read back as NaN.
 */
fa2_status fa2_kv4_append(const void* k, const void* v, const int32_t* slots, void* cache,
                          const float* k_descale, const float* v_descale, int B, int H_kv, int N, int d,
                          int64_t k_stride_b, int64_t k_stride_h, int64_t k_stride_n, int64_t v_stride_b,
                          int64_t v_stride_h, int64_t v_stride_n, int page_size, int num_pages,
                          fa2_dtype dtype, cudaStream_t stream);

/*
 * Reads cached tokens back as 16-bit tensors, for instance the context of a
 * prompt's next chunk, for fa2_fwd_ex.
 *   starts : [B] int32 or NULL (all 0): the position of row 0
 *   k, v   : [B, H_kv, N, d] (output); row i is position starts[b] + i, each
 *            value code * (scale * descale) in fp32, rounded once. Rows at or
 *            past seq_lens[b], before position 0 or on a bad page are zeros
 */
fa2_status fa2_kv4_gather(const void* cache, const int32_t* block_table, const int32_t* seq_lens,
                          const int32_t* starts, const float* k_descale, const float* v_descale, void* k,
                          void* v, int B, int H_kv, int N, int d, int max_pages, int page_size, int num_pages,
                          fa2_dtype dtype, cudaStream_t stream);

/*
 * Attention of the N_q newest tokens of each request over its cached tokens
 * (their own keys and values included, if they were appended).
 *   q, o : [B, H_q, N_q, d] 16-bit; lse : [B, H_q, N_q] fp32
 *   seq_lens : [B] int32, cached tokens of each request; 0 for an idle row
 *   causal   : 0 or 1. With 1, query row i attends position
 *              j < seq_lens[b] + i + 1 - N_q, as fa2_fwd_ex. A row with no
 *              allowed key gets O = 0 and LSE = -inf
 *   workspace : device, fa2_fwd_kv4_workspace(...) bytes (may be NULL for 0),
 *              contents irrelevant before and after; calls that may overlap
 *              need their own. After FA2_ERR_TIMEOUT it is zeroed before a
 *              captured call that uses it is replayed
 * Any N_q >= 1 is right. Up to 64 query rows a KV head (H_q / H_kv * N_q) read
 * the cache once, every 64 more once again; prompts and long chunks of them are
 * faster by fa2_kv4_gather and fa2_fwd_ex.
 * Query rows are fp16 for the products: fp16 ones as they are, bf16 ones scaled
 * by a power of two a row, exactly but for elements below 2^-31 of the row's
 * largest, which are off by 2^-39 of that at most. The softmax weights are
 * rounded to fp16 (2^-11), sums are fp32. A row of q that is not finite
 * affects no other row. A NaN in the cache affects the rows that see it.
 * B * H_q * N_q < 2^31 - 64, H_kv < 32768, and the blocks of at most 64 rows
 * of all requests and heads times max_pages * page_size / 32 up to 2^30. One
 * launch.
 */
fa2_status fa2_fwd_kv4(const void* q, const void* cache, const int32_t* block_table, const int32_t* seq_lens,
                       const float* k_descale, const float* v_descale, void* o, float* lse, void* workspace,
                       int64_t workspace_bytes, int B, int H_q, int H_kv, int N_q, int d, int max_pages,
                       int page_size, int num_pages, float scale, int causal, fa2_dtype dtype,
                       cudaStream_t stream);

/* Bytes of workspace that fa2_fwd_kv4 needs for these sizes, whatever the
 * lengths; -1 for sizes that it does not take. Not more for a smaller B,
 * max_pages or page_size. */
int64_t fa2_fwd_kv4_workspace(int B, int H_q, int H_kv, int N_q, int d, int max_pages, int page_size);

/*
 * Rotary positions with several axes (one for text; time, height and width
 * for images and video). (The source pages take q and k as they are; this
 * makes them.) Of each head's d elements the first rot_dim are rotated, as
 * rot_dim / 2 pairs: pair i is elements i and i + rot_dim / 2, or 2i and 2i + 1
 * with interleaved = 1. Its angle is positions[axes[i]][b, n] * inv_freq[i], and
 *     y1 = x1 cos - x2 sin,   y2 = x2 cos + x1 sin
 * in fp32, rounded once; elements behind rot_dim are copied. Angles are formed
 * exactly to 2^-32 of a turn for every position, far ones too (inv_freq up to 1),
 * and taken within a turn as fp32.
 *   q, q_out : [B, H_q, N, d] bf16 or fp16; k, k_out : [B, H_kv, N, d], or both
 *              NULL with H_kv = 0. Elements of a row adjacent
 *   strides  : 12 numbers in host memory, read during the call: the strides of
 *              batch entry, head and token of q, of k, of q_out and of k_out, in
 *              elements (multiples of 8, 0 .. 2^31 - 8; 0 in an output only for
 *              an axis of length 1), so that q and k may be views of a
 *              projection's output. Those of k and k_out are not read without k
 *   positions : [n_axes, B, N] int32, any value; inv_freq : [rot_dim / 2] fp32,
 *              finite; axes : [rot_dim / 2] int32 or NULL (all 0). An axis outside
 *              0 .. n_axes - 1 is reported by fa2_check_status as FA2_ERR_BOUNDS
 *              and its pair's angle is 0
 *   d : 64 or 128; rot_dim : a multiple of 16 up to d; n_axes : up to 8
 * An output may be its input (with its strides); otherwise nothing that is
 * written may overlap anything else. Pointers: tensors 16-byte aligned, others 4-byte
 * aligned. B * N < 2^31 - 1024. Errors otherwise as fa2_fwd_gqa; nothing is
 * allocated; one launch.
 */
fa2_status fa2_rope(const void* q, const void* k, void* q_out, void* k_out, const int32_t* positions,
                    const float* inv_freq, const int32_t* axes, int B, int H_q, int H_kv, int N, int d,
                    int rot_dim, int n_axes, int interleaved, const int64_t* strides, fa2_dtype dtype,
                    cudaStream_t stream);

/*
 * The gradient of fa2_rope: from those of its outputs (such as dq and dk of
 * fa2_bwd) to those of its inputs, the rotation by the opposite angles. Arguments
 * as fa2_rope, with dq_out, dk_out read and dq, dk written.
 */
fa2_status fa2_rope_bwd(const void* dq_out, const void* dk_out, void* dq, void* dk, const int32_t* positions,
                        const float* inv_freq, const int32_t* axes, int B, int H_q, int H_kv, int N, int d,
                        int rot_dim, int n_axes, int interleaved, const int64_t* strides, fa2_dtype dtype,
                        cudaStream_t stream);

/*
 * A paged KV cache in the tensors' own 16 bits. (The source pages leave the KV
 * cache out.) The cache is the caller's device memory,
 *     cache : [num_pages, H_kv, 2, page_size, d] bf16 or fp16
 * of a page and KV head first the keys of page_size tokens, then the values. A
 * token's place is its slot, page * page_size + offset; slots, block tables and
 * lengths are those of the 4-bit cache, and fa2_kv4_plan makes them for both.
 * Tokens come packed, [T, H, d], whatever requests they belong to.
 *   d : 64 or 128; page_size : 16, 32, 64 or 128; num_pages * page_size < 2^31 - 256
 * Page ids, slots, rows and lengths that point outside the cache, the table or
 * the tensors are skipped on the device and reported by fa2_check_status as
 * FA2_ERR_BOUNDS. Pointers: tensors, cache and workspace 16-byte aligned, the
 * others 4-byte aligned. Errors otherwise as fa2_fwd_gqa; nothing is allocated.
 */

/*
 * Writes new keys and values into their slots, the keys rotated on the way, and
 * rotates the queries of the same tokens.
 *   k, v     : [T, H_kv, d]; q : [T, H_q, d] or NULL with H_q = 0
 *   q_out    : [T, H_q, d] dense (output; NULL without q; may be q if that is dense)
 *   strides  : 6 numbers in host memory: the strides of token and head of q, k
 *              and v, in elements (multiples of 8, 0 .. 2^31 - 8)
 *   slots    : [T] int32; the keys and values of a negative slot are skipped, its
 *              queries are not. A slot may be named once in a call
 *   positions, inv_freq, axes, rot_dim, n_axes, interleaved : as fa2_rope, with
 *              positions [n_axes, T]; positions NULL with rot_dim = 0 and without q:
 *              keys are written as they are
 * T < 2^31 - 1024. One launch.
 */
fa2_status fa2_kv16_append(const void* q, const void* k, const void* v, const int32_t* slots,
                           const int32_t* positions, const float* inv_freq, const int32_t* axes, void* cache,
                           void* q_out, int T, int H_q, int H_kv, int d, int rot_dim, int n_axes,
                           int interleaved, const int64_t* strides, int page_size, int num_pages,
                           fa2_dtype dtype, cudaStream_t stream);

/*
 * Attention of each request's newest tokens, one or a whole chunk of a prompt,
 * over its cached tokens (their own keys and values included, if they were
 * appended). Requests of any lengths go in one call.
 *   q        : [T, H_q, d] 16-bit, of the cache's type; strides of token and
 *              head in elements (multiples of 8, 8 .. 2^31 - 8)
 *   o        : [T, H_q, d] dense; lse : [T, H_q] fp32
 *   q_starts, q_lens : [B] int32: request b's new tokens are rows q_starts[b] ..
 *              q_starts[b] + q_lens[b] - 1; 0 for an idle request. No row may belong
 *              to two. Rows of o and lse that belong to no request stay as they were
 *   seq_lens : [B] int32, cached tokens of each request
 *   block_table : [B, max_pages] int32, max_pages * page_size < 2^31 - 256; entries
 *              behind a request's last page are never read
 *   causal   : 0 or 1. With 1, new token i of request b attends position
 *              j < seq_lens[b] + i + 1 - q_lens[b]. A row with no allowed key gets
 *              O = 0 and LSE = -inf
 *   workspace : device, fa2_fwd_kv16_workspace(...) bytes, contents irrelevant
 *              before and after; calls that may overlap need their own
 * Query heads that share a KV head: up to 128. Both products take 16-bit operands:
 * the softmax's weights are rounded to the cache's type (bf16 2^-8, fp16 2^-11);
 * scores, sums and partial results are fp32. What lies in a request's pages behind
 * its last token has no effect, whatever it is. A key or value that is not finite
 * affects the rows that see it, a row of q that is not finite itself alone. An infinite
 * value gives such a row that infinity, whatever the chunk (NaN with one of the
 * other sign or a NaN beside it; and NaN may stand for an infinity whose weight
 * rounds to zero). A row whose allowed scores are all -inf is as one without a
 * key. A page that is skipped reads as zeros.
 * T * H_q < 2^31, num_pages * H_kv < 2^30 - 1, and H_kv times the blocks of 256 query
 * rows (T tokens fill 256 / (H_q / H_kv) of them each, one more a request) times
 * (4 + 3 tiles of 128 keys of a full table) up to 2^30. Two launches.
 */
fa2_status fa2_fwd_kv16(const void* q, const void* cache, const int32_t* block_table, const int32_t* seq_lens,
                        const int32_t* q_starts, const int32_t* q_lens, void* o, float* lse, void* workspace,
                        int64_t workspace_bytes, int T, int B, int H_q, int H_kv, int d, int64_t q_stride_t,
                        int64_t q_stride_h, int max_pages, int page_size, int num_pages, float scale, int causal,
                        fa2_dtype dtype, cudaStream_t stream);

/* Bytes of workspace that fa2_fwd_kv16 needs for these sizes, whatever the
 * lengths; -1 for sizes that it does not take. */
int64_t fa2_fwd_kv16_workspace(int T, int B, int H_q, int H_kv, int d, int max_pages, int page_size);

/*
 * Synchronises `stream`, then reads and clears the status word of the device
 * that `stream` belongs to (the current device is switched to it for the
 * read and restored afterwards). Returns FA2_ERR_TIMEOUT if a kernel since
 * the last check abandoned a wait (its outputs are then undefined),
 * FA2_ERR_BOUNDS if a device-side bounds check failed (the KV cache's checks
 * are in every build, all others in debug builds only),
 * FA2_ERR_CUDA if the stream reported an error, FA2_OK otherwise.
 * There is one status word per device, shared by every stream and host
 * thread that uses the device: a timeout of a kernel on another stream is
 * reported to whichever caller checks first (and then cleared), and a kernel
 * still running on another stream may set the word after this call read it.
 * Callers that need per-stream attribution check after synchronising all
 * streams that ran the library's kernels.
 */
fa2_status fa2_check_status(cudaStream_t stream);

/* Human-readable name of a status code (static storage, never NULL). */
const char* fa2_status_string(fa2_status status);

/*
 * Watchdog limit for each in-kernel wait, in nanoseconds, for kernels
 * launched after the call on any device of this process (default 2e9, i.e.
 * two seconds; values <= 0 restore the default). Returns the previous value.
 */
int64_t fa2_set_wait_limit_ns(int64_t limit_ns);

/*
 * Test hook for the watchdog. With flags = 1 the next 16-bit forward kernels
 * and the backward's dK/dV kernel skip the load of their query tiles, and the
 * KV cache's kernel for more than 24 query rows that of its keys, so their
 * waits run out and the status word reports
 * FA2_ERR_TIMEOUT; the kernel still frees its tensor memory, waits for its
 * own copies and returns normally. 0 (the default) restores normal
 * operation. Returns the previous flags.
 */
int fa2_set_debug_flags(int flags);

/*
 * The planner's kernel choice where two kernels compute the same result
 * (process-wide, for calls made after it returns). Bit 0 (value 1): d = 64
 * with equal lengths runs the 16-bit kernel's d = 64 path (P written over S,
 * one MMA-issuing warp) instead of the default d = 64 kernel (P in TMEM
 * columns of its own, separate warps for Q K^T and P V), which measured
 * faster. Results differ only by rounding order and are within the same
 * tolerance. The first call to the library reads the initial value from the
 * environment: FA2_TILE_CFG=d64=shared sets bit 0, anything else or no
 * variable gives 0. Returns the previous value, or -1 (nothing changed) if
 * config is negative or has a bit other than bit 0 set.
 */
int fa2_set_tile_config(int config);

/* Library version string, e.g. "fa2-sm103a 0.5.0" ("... debug" for the
 * FA2_DEBUG build, libfa2_debug.so). */
const char* fa2_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FA2_H_ */
