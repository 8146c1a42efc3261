/*
 * kvstore.h -- C ABI of the GB300 (sm_103a) KV-cache write library.
 *
 * For every new token t, the K row and the V row (num_heads x head_dim
 * elements, arbitrary byte strides) are written into row indices[t] of a
 * large K cache and V cache:
 *
 *   kv_store      plain byte-exact copy of the rows;
 *   kv_store_fp8  each element is widened to fp32, optionally multiplied by a
 *                 per-tensor fp32 inverse scale, converted to FP8 e4m3fn and
 *                 written at the paged cache address of the slot.
 *
 * Sources (sglang): kvcache.cuh, kernel `store_kvcache` and host launcher
 * `StoreKVCacheKernel::run` (plain copy, the row-split option and the slot
 * bound 0 <= slot < size_limit); trtllm_fp8_kv_kernel.py, kernels
 * `_fused_fp8_set_kv_buffer_kernel` / `_process_kv_tensor` and the wrapper
 * `fused_fp8_set_kv_buffer` (page decomposition, strides, fp32 inverse scale
 * read on the device, e4m3fn conversion).
 *
 * Conventions shared by every call:
 *  - All tensor pointers are memory owned by the caller; the library never
 *    allocates, frees or retains them, and never allocates memory of its own
 *    during a call.  Caches and error records are device memory
 *    (kv_error_snapshot may also write to page-locked host memory).  The
 *    token-major side of every call -- the inputs of the writes (k, v) and
 *    the outputs of the gathers (k_out, v_out) -- and the slot ids may also
 *    be page-locked host memory (cudaHostAlloc / cudaHostRegister), which the
 *    kernels read or write in place over NVLink-C2C or PCIe.  Pointers CUDA
 *    does not know (pageable host memory, stray addresses) are rejected with
 *    KV_ERR_INVALID_ARG before anything is launched.
 *  - Calls are asynchronous on `stream` and do not synchronise the host,
 *    except kv_error_poll.  They may be captured in a CUDA graph.
 *  - Every kernel launched here waits for the work that precedes it on the
 *    stream before it touches memory (programmatic dependent launch), so the
 *    stream's ordering is kept.
 *  - Strides are in BYTES and may be any int64 value; elements of one head
 *    are contiguous when the dim stride equals the element size, which is the
 *    fast path.  Bases and strides that are not 16-byte multiples select
 *    narrower vector widths; this is never an error.
 *  - An out-of-range slot (outside [0, size_limit)) is not an argument error:
 *    the kernel skips that token (neither its K nor its V row is written),
 *    counts it in the caller's error record and continues.  kv_error_poll
 *    reports it.  No slot value can cause a write outside the rows
 *    [0, size_limit) of the caches.
 *  - size_limit is trusted to be at most the number of cache rows.
 *  - Duplicate slots: calls write the candidate rows concurrently, so each
 *    element of such a cache row equals the same element of one of the
 *    candidate rows; which candidate is unspecified and may differ from
 *    element to element (and between the K and the V row).
 *  - The inputs and the index array must not overlap the caches.
 *  - num_tokens == 0 returns KV_OK without launching (pointers may be NULL).
 */
#ifndef FP8_QUANT_GB300_KVSTORE_H
#define FP8_QUANT_GB300_KVSTORE_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define KV_ABI_VERSION 1

/* Same type as cudaStream_t.  NULL selects the legacy default stream. */
typedef struct CUstream_st *kv_stream_t;

typedef enum kv_status {
    KV_OK = 0,
    KV_ERR_INVALID_ARG = 1,  /* bad argument found on the host; nothing was launched */
    KV_ERR_UNSUPPORTED = 2,  /* legal request this library does not implement; nothing launched */
    KV_ERR_CUDA = 3,         /* a CUDA runtime call failed; see kv_last_cuda_error() */
    KV_ERR_INDEX_OOB = 4,    /* kv_error_poll: at least one token had an out-of-range slot */
    KV_ERR_WAIT = 5          /* kv_error_poll: a kernel gave up a wait; outputs of its call are not to be used */
} kv_status;

typedef enum kv_index_dtype { KV_INDEX_I32 = 0, KV_INDEX_I64 = 1 } kv_index_dtype;

/* Element type of the K/V inputs of kv_store_fp8 (2-byte floats). */
typedef enum kv_src_dtype { KV_SRC_F16 = 0, KV_SRC_BF16 = 1 } kv_src_dtype;

/* Byte strides.  Element (t, h, d) of K is at k + t*k_token + h*k_head +
 * d*k_dim; element (h, d) of cache row s is at k_cache + s*kc_slot +
 * h*kc_head + d*kc_dim (kv_store_fp8 adds the page decomposition, below).
 * The K cache and the V cache have separate strides. */
typedef struct kv_strides {
    int64_t k_token, k_head, k_dim;
    int64_t v_token, v_head, v_dim;
    int64_t kc_slot, kc_head, kc_dim;
    int64_t vc_slot, vc_head, vc_dim;
} kv_strides;

/* Device-side error record, owned by the caller (16 bytes, 8-byte aligned,
 * zero-initialised before first use, e.g. with cudaMemsetAsync or
 * kv_error_reset).  Kernels only add to it; kv_error_poll reads and clears it.
 * Calls that share one record on different streams share its counts. */
#define KV_ERROR_WAIT_BIT (1ull << 63)
typedef struct kv_error_record {
    uint64_t oob_count;      /* tokens skipped because their slot was out of range; KV_ERROR_WAIT_BIT
                              * beside them when a kernel of kv_attend gave up a wait */
    uint64_t first_bad_key;  /* bitwise NOT of the lowest skipped token; 0 if none */
} kv_error_record;

/*
 * kv_store -- plain copy (sglang kvcache.cuh, `store_kvcache`).
 *
 *   k, v           device pointers to element (0, 0, 0) of the K and V inputs.
 *   k_cache,
 *   v_cache        device pointers to element (slot 0, 0, 0) of the caches.
 *   indices        device pointer to num_tokens slot ids (int32 or int64 per
 *                  index_dtype), read at indices[t * index_stride]
 *                  (index_stride in ELEMENTS, >= 1).
 *   num_heads,
 *   head_dim       row shape, both >= 1.
 *   elem_bytes     element size: 1, 2, 4 or 8 (the copy is byte-exact, so the
 *                  element type does not matter; bf16/fp16 rows use 2).
 *   strides        byte strides (host pointer, read during the call only).
 *   size_limit     slots must satisfy 0 <= slot < size_limit.
 *   num_split      how many parts each contiguous row is split into, each
 *                  part copied by its own warp: 0 = choose automatically,
 *                  1, 2 or 4.  2 and 4 need the row's bytes (num_heads *
 *                  head_dim * elem_bytes) to be a multiple of 256 and 512
 *                  respectively (the split rule of `StoreKVCacheKernel`);
 *                  otherwise KV_ERR_INVALID_ARG.  The result does not depend
 *                  on num_split.
 *   d_err          device error record (required when num_tokens > 0).
 *   stream         CUDA stream.
 *
 * Returns KV_OK once the kernel is enqueued, KV_ERR_INVALID_ARG for a bad
 * argument (NULL pointer, num_tokens < 0, num_heads/head_dim < 1, bad
 * elem_bytes, index_dtype, index_stride, num_split or split rule, size_limit
 * < 0, misaligned d_err), KV_ERR_CUDA if the launch failed.
 */
kv_status kv_store(const void *k, const void *v, void *k_cache, void *v_cache,
                   const void *indices, kv_index_dtype index_dtype, int64_t index_stride,
                   int64_t num_tokens, int32_t num_heads, int32_t head_dim,
                   int32_t elem_bytes, const kv_strides *strides, int64_t size_limit,
                   int32_t num_split, kv_error_record *d_err, kv_stream_t stream);

/*
 * kv_store_paged -- kv_store into a paged cache [pages, page_size, H, D]
 * whose page stride may include padding: slot s is written at
 * (s / page_size) * kc_page_stride + (s % page_size) * kc_slot + h * kc_head
 * + d * kc_dim (likewise for V), the 4-D write of trtllm_fp8_kv_kernel.py
 * `_naive_fp8_set_kv_buffer` (k_cache[page_ids, page_offsets] = k) for a
 * cache of the input's own type.  A page stride of page_size * kc_slot is
 * the flat layout of kv_store.  Other arguments and errors as kv_store, plus
 * KV_ERR_INVALID_ARG for page_size < 1.
 */
kv_status kv_store_paged(const void *k, const void *v, void *k_cache, void *v_cache,
                         const void *indices, kv_index_dtype index_dtype, int64_t index_stride,
                         int64_t num_tokens, int32_t num_heads, int32_t head_dim,
                         int32_t elem_bytes, const kv_strides *strides, int64_t page_size,
                         int64_t kc_page_stride, int64_t vc_page_stride, int64_t size_limit,
                         int32_t num_split, kv_error_record *d_err, kv_stream_t stream);

/*
 * kv_store_fp8 -- fused scale + FP8 e4m3fn conversion + paged write
 * (sglang trtllm_fp8_kv_kernel.py, `_fused_fp8_set_kv_buffer_kernel`,
 * `_process_kv_tensor`, wrapper `fused_fp8_set_kv_buffer`).
 *
 * Arguments as for kv_store, except:
 *   k, v           bf16 or fp16 inputs (src_dtype); addresses and the
 *                  k/v strides must be even.
 *   k_cache,
 *   v_cache        caches of e4m3fn bytes (kc_dim / vc_dim are the byte
 *                  distance between consecutive dims, normally 1).
 *   page_size      tokens per page, >= 1.  Slot s is written at
 *                  (s / page_size) * kc_page_stride + (s % page_size) * kc_slot
 *                  + h * kc_head + d * kc_dim (likewise for V).  A 3-D cache
 *                  [slots, H, D] passes kc_page_stride = page_size * kc_slot,
 *                  which makes this s * kc_slot; a 4-D cache
 *                  [pages, page_size, H, D] passes its page stride.
 *   inv_k_scale,
 *   inv_v_scale    DEVICE pointers to one fp32 each (the inverse scales),
 *                  read by the kernel, so no host synchronisation is needed;
 *                  both must be non-NULL when use_scale != 0 and are ignored
 *                  otherwise.
 *   use_scale      0: convert x unscaled; else convert fl32(x * inv).
 *
 * Numerics (per element): x is widened exactly to fp32; y = x * inv in fp32
 * with round-to-nearest-even (no fused operations, denormals kept); the code
 * is the e4m3fn value nearest to y, ties to the even mantissa, with finite
 * overflow and +-Inf saturated to +-448 and every NaN written as 0x7F.
 * use_scale == 0 gives the same bytes as use_scale != 0 with inv = 1.0f.
 *
 * Returns as kv_store; KV_ERR_INVALID_ARG also for a bad src_dtype,
 * page_size < 1, odd input addresses or strides, or a NULL scale pointer
 * with use_scale != 0.
 */
kv_status kv_store_fp8(const void *k, const void *v, void *k_cache, void *v_cache,
                       const void *indices, kv_index_dtype index_dtype, int64_t index_stride,
                       int64_t num_tokens, int32_t num_heads, int32_t head_dim,
                       kv_src_dtype src_dtype, const kv_strides *strides, int64_t page_size,
                       int64_t kc_page_stride, int64_t vc_page_stride, int64_t size_limit,
                       const float *inv_k_scale, const float *inv_v_scale, int32_t use_scale,
                       kv_error_record *d_err, kv_stream_t stream);

/*
 * kv_gather -- the inverse of kv_store: row t of k_out / v_out takes the cache
 * row of slot indices[t], byte for byte.  The single-GPU counterpart of the
 * materialise step of vLLM dcp_direct_kv_gather.cu
 * (`materialize_kv_gather_kernel`), and the read-back half of a round trip.
 *
 * Arguments as for kv_store with the roles of the tensors swapped: k_cache /
 * v_cache are read, k_out / v_out are written.  In `strides`, k_* / v_*
 * describe the OUTPUT rows and kc_* / vc_* the caches.  An out-of-range slot
 * leaves output row t untouched and is counted in d_err.  The outputs must
 * not overlap the caches or the indices.
 */
kv_status kv_gather(const void *k_cache, const void *v_cache, void *k_out, void *v_out,
                    const void *indices, kv_index_dtype index_dtype, int64_t index_stride,
                    int64_t num_tokens, int32_t num_heads, int32_t head_dim,
                    int32_t elem_bytes, const kv_strides *strides, int64_t size_limit,
                    kv_error_record *d_err, kv_stream_t stream);

/*
 * kv_gather_paged -- kv_gather from a paged cache [pages, page_size, H, D]
 * (the inverse of kv_store_paged): slot s is read at
 * (s / page_size) * kc_page_stride + (s % page_size) * kc_slot + ... .
 * Other arguments and errors as kv_gather, plus KV_ERR_INVALID_ARG for
 * page_size < 1.
 */
kv_status kv_gather_paged(const void *k_cache, const void *v_cache, void *k_out, void *v_out,
                          const void *indices, kv_index_dtype index_dtype, int64_t index_stride,
                          int64_t num_tokens, int32_t num_heads, int32_t head_dim,
                          int32_t elem_bytes, const kv_strides *strides, int64_t page_size,
                          int64_t kc_page_stride, int64_t vc_page_stride, int64_t size_limit,
                          kv_error_record *d_err, kv_stream_t stream);

/*
 * kv_gather_fp8 -- dequantising gather from e4m3fn caches written by
 * kv_store_fp8 (same page addressing: page_size, kc_page_stride,
 * vc_page_stride).  Each code is decoded exactly to fp32, multiplied by the
 * fp32 scale (k_scale / v_scale: DEVICE pointers, the forward scales, i.e.
 * 1/inv) when use_scale != 0, and rounded to nearest-even bf16 or fp16
 * (out_dtype).  NaN codes become the canonical NaN 0x7FFF; fp16 overflow
 * becomes +-Inf.  Output strides (k_* / v_*) must be even.
 */
kv_status kv_gather_fp8(const void *k_cache, const void *v_cache, void *k_out, void *v_out,
                        const void *indices, kv_index_dtype index_dtype, int64_t index_stride,
                        int64_t num_tokens, int32_t num_heads, int32_t head_dim,
                        kv_src_dtype out_dtype, const kv_strides *strides, int64_t page_size,
                        int64_t kc_page_stride, int64_t vc_page_stride, int64_t size_limit,
                        const float *k_scale, const float *v_scale, int32_t use_scale,
                        kv_error_record *d_err, kv_stream_t stream);

/* FP8 cache formats of the extended calls. */
typedef enum kv_fp8_format {
    KV_FP8_E4M3FN = 0,   /* largest finite 448, no infinities */
    KV_FP8_E5M2 = 1      /* largest finite 57344 */
} kv_fp8_format;

/* Scale modes of the extended calls. */
typedef enum kv_scale_mode {
    KV_SCALE_NONE = 0,        /* values converted unscaled */
    KV_SCALE_TENSOR = 1,      /* one fp32 scale per tensor, a device scalar */
    KV_SCALE_TOKEN = 2,       /* one scale per token row (all heads), computed per call */
    KV_SCALE_TOKEN_HEAD = 3,  /* one scale per (token, head), computed per call */
    KV_SCALE_PAGE = 4         /* one fp32 scale per cache page, supplied by the caller */
} kv_scale_mode;

/*
 * kv_store_fp8_ex -- kv_store_fp8 with a choice of FP8 format and of scale
 * granularity, including scales computed in the kernel.  The fused FP8
 * write's module docstring (trtllm_fp8_kv_kernel.py) names per-token scale
 * computation and e5m2 caches; its kernel implements the per-tensor e4m3fn
 * case only, which is kv_store_fp8 (= this call with KV_FP8_E4M3FN and
 * KV_SCALE_TENSOR or KV_SCALE_NONE).
 *
 * Arguments as kv_store_fp8, plus:
 *   format       KV_FP8_E4M3FN or KV_FP8_E5M2 (rounding: nearest even; finite
 *                overflow and infinities saturate to the largest finite
 *                value; every NaN becomes 0x7F).
 *   scale_mode   KV_SCALE_NONE / KV_SCALE_TENSOR: as kv_store_fp8 with
 *                use_scale 0 / 1 (inv_k_scale, inv_v_scale are device
 *                pointers to the inverse scales).
 *                KV_SCALE_TOKEN / KV_SCALE_TOKEN_HEAD: for each group (the
 *                token's K row or V row, or one head of it) the kernel takes
 *                amax = max |x| (NaN ignored), inv = fmax / amax and
 *                scale = amax / fmax in fp32 round-to-nearest (both 1 when
 *                amax is 0; fmax = 448 or 57344), writes the codes of
 *                fl32(x * inv), and stores `scale` (the dequantisation
 *                multiplier) at k_scales[slot * scales_slot_stride + g],
 *                g = head (TOKEN_HEAD) or 0 (TOKEN); likewise V.  The scale
 *                caches are device float arrays indexed by slot, not by page.
 *                KV_SCALE_PAGE: inv_k_scale / inv_v_scale point to device
 *                arrays of fp32 INVERSE scales, one per cache page; the
 *                token written to slot s uses inv[s / page_size] in place of
 *                the per-tensor scalar (codes of fl32(x * inv[s / page_size])).
 *                The arrays must hold ceil(size_limit / page_size) floats.
 *                The fused FP8 write's module docstring names per-page scales
 *                and its kernel has none; the page is the one its kernel
 *                computes, slot // page_size.  Any layout kv_store_fp8 takes.
 *   k_scales,
 *   v_scales,
 *   scales_slot_stride   used by the dynamic modes only: non-NULL, 4-byte
 *                aligned, stride >= num_heads (TOKEN_HEAD) or >= 1 (TOKEN).
 * The dynamic modes need contiguous dims (k_dim = v_dim = 2, kc_dim = vc_dim
 * = 1), else KV_ERR_UNSUPPORTED.  Out-of-range slots write neither codes nor
 * scales.
 */
kv_status kv_store_fp8_ex(const void *k, const void *v, void *k_cache, void *v_cache,
                          const void *indices, kv_index_dtype index_dtype, int64_t index_stride,
                          int64_t num_tokens, int32_t num_heads, int32_t head_dim,
                          kv_src_dtype src_dtype, const kv_strides *strides, int64_t page_size,
                          int64_t kc_page_stride, int64_t vc_page_stride, int64_t size_limit,
                          kv_fp8_format format, kv_scale_mode scale_mode,
                          const float *inv_k_scale, const float *inv_v_scale, float *k_scales,
                          float *v_scales, int64_t scales_slot_stride, kv_error_record *d_err,
                          kv_stream_t stream);

/*
 * kv_gather_fp8_ex -- kv_gather_fp8 for every layout kv_store_fp8_ex writes:
 * codes of `format` decoded exactly, multiplied by the scale of `scale_mode`
 * (NONE: none; TENSOR: *k_scale / *v_scale, the forward scales; TOKEN /
 * TOKEN_HEAD: k_scales[slot * scales_slot_stride + g] as written by
 * kv_store_fp8_ex; PAGE: k_scale[slot / page_size] / v_scale[...], device
 * arrays of forward scales, one per cache page), rounded to bf16 / fp16.
 * kv_gather_fp8 is this call with KV_FP8_E4M3FN and NONE / TENSOR.
 */
kv_status kv_gather_fp8_ex(const void *k_cache, const void *v_cache, void *k_out, void *v_out,
                           const void *indices, kv_index_dtype index_dtype, int64_t index_stride,
                           int64_t num_tokens, int32_t num_heads, int32_t head_dim,
                           kv_src_dtype out_dtype, const kv_strides *strides, int64_t page_size,
                           int64_t kc_page_stride, int64_t vc_page_stride, int64_t size_limit,
                           kv_fp8_format format, kv_scale_mode scale_mode, const float *k_scale,
                           const float *v_scale, const float *k_scales, const float *v_scales,
                           int64_t scales_slot_stride, kv_error_record *d_err,
                           kv_stream_t stream);

/*
 * kv_inv_scale -- inv[i] = 1 / scale[i] in fp32, round to nearest, for
 * i < n, on the device (trtllm_fp8_kv_kernel.py, `fused_fp8_set_kv_buffer`
 * forms 1.0 / k_scale on the GPU so that graph capture needs no host sync).
 * scale and inv are device pointers to n floats (4-byte aligned; they may be
 * the same array).  n == 0: KV_OK, nothing launched.
 */
kv_status kv_inv_scale(const float *scale, float *inv, int64_t n, kv_stream_t stream);

/*
 * kv_absmax_inv -- per-tensor scale of the K rows and of the V rows on the
 * device: amax[0] = max |K|, amax[1] = max |V| over all num_tokens x num_heads
 * x head_dim elements (NaN elements ignored; 0 for an empty or all-NaN
 * tensor), and inv[j] = fp8_max / amax[j] in fp32 round-to-nearest (1.0 when
 * amax[j] is 0).  With fp8_max = 448 this is the per-tensor inverse scale
 * kv_store_fp8 takes (e4m3fn's largest finite value maps to the tensor's
 * largest magnitude).
 *   k, v       bf16 / fp16 rows (src_dtype); strides->k_* and v_* are used
 *              (dims must be contiguous: k_dim = v_dim = 2; else
 *              KV_ERR_UNSUPPORTED).
 *   amax, inv  device pointers to two floats each, written by the call.
 *   work       NULL, or a device workspace of KV_ABSMAX_WORK_BYTES (4-byte
 *              aligned) owned by the caller: zero before its first use (e.g.
 *              cudaMemsetAsync), and left zero by every call that completes.
 *              With it a call is two kernels (reduce, finish); without it,
 *              three (amax is cleared by a kernel first and serves as the
 *              accumulator).  Calls that share one workspace must not
 *              overlap on the GPU (their maxima would mix); calls on one
 *              stream never do.
 * fp8_max must be positive and finite.
 */
#define KV_ABSMAX_WORK_BYTES 8
kv_status kv_absmax_inv(const void *k, const void *v, kv_src_dtype src_dtype,
                        int64_t num_tokens, int32_t num_heads, int32_t head_dim,
                        const kv_strides *strides, float fp8_max, float *amax, float *inv,
                        uint32_t *work, kv_stream_t stream);

/*
 * kv_store_fp8_dynamic_tensor -- the FP8 write with per-tensor scales formed
 * from the batch itself, in one call: the fused form of kv_absmax_inv
 * followed by kv_store_fp8_ex in KV_SCALE_TENSOR mode (the trtllm page's
 * docstring advertises computed scales while its kernel takes a given one;
 * the recipe is the per-tensor one, inv = fmax / amax).
 *   amax_k = max |K| and amax_v = max |V| over all num_tokens rows (NaN
 *   elements ignored; out-of-range slots do not exclude their rows), then
 *   inv = fmax / amax in fp32 round-to-nearest (1.0 when amax is 0) and the
 *   codes fp8(fl32(x * inv)) as kv_store_fp8_ex writes them; fmax is 448
 *   (e4m3fn) or 57344 (e5m2).  *k_scale / *v_scale receive the forward
 *   (dequantisation) scales amax / fmax (1.0 when amax is 0), what
 *   kv_gather_fp8_ex takes in KV_SCALE_TENSOR mode.
 * Arguments as kv_store_fp8_ex, plus:
 *   k_scale, v_scale  device pointers to one float each (4-byte aligned).
 *   work   device workspace of KV_DYNAMIC_TENSOR_WORK_BYTES (8-byte aligned),
 *          owned by the caller, zero before its first use.  It holds a
 *          generation counter and the two maxima tagged with it, so a call
 *          needs no clearing pass: two kernels (the reduction, then the
 *          write, which forms the inverse scales in its prologue).  Calls
 *          sharing one workspace must not overlap on the GPU; calls on one
 *          stream never do.  After a KV_ERR_CUDA return its contents are
 *          undefined: zero it again before the next call.
 * Dims must be contiguous on the input side (k_dim = v_dim = 2; else
 * KV_ERR_UNSUPPORTED); the cache side may use any layout kv_store_fp8_ex
 * takes.  num_tokens == 0: KV_OK, nothing launched, nothing written.
 */
#define KV_DYNAMIC_TENSOR_WORK_BYTES 24
kv_status kv_store_fp8_dynamic_tensor(const void *k, const void *v, void *k_cache,
                                      void *v_cache, const void *indices,
                                      kv_index_dtype index_dtype, int64_t index_stride,
                                      int64_t num_tokens, int32_t num_heads, int32_t head_dim,
                                      kv_src_dtype src_dtype, const kv_strides *strides,
                                      int64_t page_size, int64_t kc_page_stride,
                                      int64_t vc_page_stride, int64_t size_limit,
                                      kv_fp8_format format, float *k_scale, float *v_scale,
                                      uint64_t *work, kv_error_record *d_err, kv_stream_t stream);

/* Formats of a KV cache that is written with the position rotation and read by
 * attention. */
typedef enum kv_cache_format {
    KV_CACHE_SRC = 0,      /* elements of the source type (2 bytes) */
    KV_CACHE_E4M3FN = 1,   /* one e4m3fn byte per element, an fp32 scale per tensor */
    KV_CACHE_E2M1 = 2      /* 4 bits per element, an e4m3fn scale per 16 dims, an fp32 scale per tensor */
} kv_cache_format;

/* The block scales of an e2m1 cache (byte strides).  A head row of head_dim
 * elements is head_dim / 2 bytes of codes, dim 2j in the low and dim 2j + 1 in
 * the high half of byte j, and head_dim / 16 e4m3fn bytes; the scale of dims
 * 16j .. 16j + 15 of (slot s, head h) is the byte at
 * k + (s / page_size) * k_page + (s % page_size) * k_slot + h * k_head + j
 * (likewise v).  An element's value is code * block scale * tensor scale. */
#define KV_FP4_BLOCK 16
typedef struct kv_block_scales {
    void *k, *v;
    int64_t k_page, k_slot, k_head;
    int64_t v_page, v_slot, v_head;
} kv_block_scales;

/* The position rotation of kv_store_rope (host struct, read during the call
 * only). */
typedef struct kv_rope {
    const float *cos_sin;       /* device: row p holds cos(a_0 .. a_{R/2-1}), then the sines; R = rotary_dim
                                 * (NULL when R is 0) */
    int64_t cos_sin_stride;     /* floats between rows, >= rotary_dim */
    int64_t max_position;       /* rows of the table; positions must satisfy 0 <= p < max_position */
    const void *positions;      /* token t's position is positions[t * position_stride] */
    kv_index_dtype position_dtype;
    int64_t position_stride;    /* in elements, >= 1 */
    int32_t rotary_dim;         /* R: even, 0 <= R <= head_dim; dims from R on are not rotated */
    int32_t interleaved;        /* 0: pairs (i, i + R/2); else pairs (2i, 2i + 1) */
    const void *q;              /* optional query rows [num_tokens, num_q_heads, head_dim], NULL: none */
    void *q_out;                /* their rotated form (may be q itself, with q's strides) */
    int32_t num_q_heads;
    int64_t q_token, q_head, qo_token, qo_head;  /* byte strides; dims contiguous */
} kv_rope;

/*
 * kv_store_rope -- append K and V rows to a paged cache with the position
 * rotation applied on the way, and rotate the query rows of the same tokens.
 * The pages write rows that something else has rotated; this call saves that
 * pass over K and Q.
 *
 * For token t with position p, each pair (a, b) of the first rotary_dim dims
 * of every K and Q head becomes
 *     a' = fl(fl(a c) - fl(b s)),   b' = fl(fl(b c) + fl(a s)),
 * c = cos_sin[p][i], s = cos_sin[p][R/2 + i], in fp32 (each operation rounded
 * to nearest); V and the dims from R on are taken as they are.  Then
 *   KV_CACHE_SRC     the value is rounded once to the source type (V and
 *                    unrotated dims keep their bytes; the sign or payload of a
 *                    NaN that is rotated is not kept);
 *   KV_CACHE_E4M3FN  the code of fl(x * inv) is written as in kv_store_fp8;
 *   KV_CACHE_E2M1    y = fl(x * inv); per block of 16 dims
 *                    S = e4m3fn(fl(max|y| * fl(1/6))) (NaN ignored, saturating
 *                    at 448), r = fl(1 / S) (0 when S is 0), and the code of
 *                    fl(y * r): nearest, ties to the even code, saturating at
 *                    +-6; every NaN is written as +6.
 * inv is *inv_k_scale / *inv_v_scale (device scalars), or 1 where the pointer
 * is NULL; KV_CACHE_SRC takes none.  Q is rounded once to the source type.
 *
 * Arguments as kv_store_fp8, plus:
 *   rope     see above.  With q set, q_out is written for every token whose
 *            position is in range, also where its slot is not.
 *   format   of the caches; KV_CACHE_E2M1 needs `scales` and head_dim a
 *            multiple of 16.
 * A token whose position is out of range writes nothing and is counted in the
 * error record once, like one whose slot is.
 * K, V, Q, q_out, the slot ids and the positions may be page-locked host
 * memory; the caches, scales, the table and the record are device memory.  Any
 * that CUDA does not know is rejected with KV_ERR_INVALID_ARG.
 * q_out may be q; it must overlap nothing else.  Dims of Q must be contiguous;
 * K, V and the caches may have any dim strides, but an e2m1 cache and its
 * scales have contiguous dims (else KV_ERR_UNSUPPORTED).  Of tokens that share a
 * slot, an e2m1 block's codes and its scale may be different ones'.
 */
kv_status kv_store_rope(const void *k, const void *v, void *k_cache, void *v_cache,
                        const void *indices, kv_index_dtype index_dtype, int64_t index_stride,
                        int64_t num_tokens, int32_t num_heads, int32_t head_dim,
                        kv_src_dtype src_dtype, const kv_strides *strides, int64_t page_size,
                        int64_t kc_page_stride, int64_t vc_page_stride, int64_t size_limit,
                        const kv_rope *rope, kv_cache_format format, const float *inv_k_scale,
                        const float *inv_v_scale, const kv_block_scales *scales,
                        kv_error_record *d_err, kv_stream_t stream);

/*
 * kv_gather_fp4 -- dequantising gather from e2m1 caches written by
 * kv_store_rope: row t of k_out / v_out takes fl16(fl(code * S * scale)) of the
 * cache row of slot indices[t] (code * S is exact in fp32; scale is *k_scale /
 * *v_scale, forward scales in device memory, or 1 where the pointer is NULL).
 * A NaN block scale (code 0x7F or 0xFF; never written by kv_store_rope) gives
 * the canonical NaN 0x7FFF.  Other arguments and errors as kv_gather_fp8;
 * kc_dim and vc_dim are not used (a row's codes are contiguous), the output's
 * dims must be (else KV_ERR_UNSUPPORTED).
 */
kv_status kv_gather_fp4(const void *k_cache, const void *v_cache, const kv_block_scales *scales,
                        void *k_out, void *v_out, const void *indices,
                        kv_index_dtype index_dtype, int64_t index_stride, int64_t num_tokens,
                        int32_t num_heads, int32_t head_dim, kv_src_dtype out_dtype,
                        const kv_strides *strides, int64_t page_size, int64_t kc_page_stride,
                        int64_t vc_page_stride, int64_t size_limit, const float *k_scale,
                        const float *v_scale, kv_error_record *d_err, kv_stream_t stream);

/* Byte strides of kv_attend.  Element (t, h, d) of q is at q + t * q_token +
 * h * q_head + d * 2 (likewise out); cache row (page, offset, head) starts at
 * k_cache + page * kc_page + offset * kc_slot + head * kc_head. */
typedef struct kv_attend_strides {
    int64_t q_token, q_head;
    int64_t o_token, o_head;
    int64_t kc_page, kc_slot, kc_head;
    int64_t vc_page, vc_slot, vc_head;
} kv_attend_strides;

/*
 * kv_attend -- softmax attention of ragged queries over a paged cache, causal,
 * with an optional sliding window and a number of first tokens (sinks) that
 * stay visible.
 *
 * Sequence b has seq_lens[b] tokens in the cache, token j at offset
 * j % page_size of page page_table[b * table_stride + j / page_size], and the
 * query rows q_start[b] .. q_start[b + 1] - 1 (q_start NULL: row b alone).
 * They are its newest tokens: query i of n_q stands at position
 * p = seq_lens[b] - n_q + i, and sees key j when
 *     0 <= j <= p  and  (window == 0  or  j > p - window  or  j < sinks).
 * Query head h reads KV head h / (num_q_heads / num_heads):
 *     s_j = sm_scale * k_scale * sum_d q_d k_jd,
 *     out = v_scale * sum_j exp(s_j) v_j / sum_j exp(s_j),
 *     lse = log sum_j exp(s_j)  (natural logarithm),
 * over the visible keys.  A row that sees no key is 0 with lse -infinity.
 * Statistics and sums are fp32; 16-bit caches are multiplied in their type,
 * e4m3fn and e2m1 values (with their block scales, both exact) in fp16 against
 * queries brought into fp16's range by a power of two per row.  The weights
 * exp(s_j) meet the values as 16-bit operands (fp16, or bf16 for a bf16 cache):
 * rounded once in the kernel for many query rows and for quantised caches, as
 * two terms (no loss beside the output's rounding) for few rows over a 16-bit
 * cache, and kept in fp32 by the general kernel.  One rounding adds up to
 * 2^-9 (bf16) or 2^-12 (fp16) of sum p_j |v_j| / sum p_j to the output's error.
 *
 *   q, out      [num_q_tokens, num_q_heads, head_dim] of `dtype`; out must not
 *               overlap q or the caches.
 *   lse         NULL, or device floats [num_q_tokens, num_q_heads], contiguous.
 *   page_table  int32 device array, table_width entries per sequence, rows
 *               table_stride (>= table_width) entries apart.
 *   seq_lens    int32 device array [num_seqs].
 *   q_start     NULL (then num_q_tokens == num_seqs), or int32 device array
 *               [num_seqs + 1], non-decreasing; values are clamped to
 *               [0, num_q_tokens], rows outside every range are not written.
 *   num_pages   pages of the caches.  Keys of a page id outside
 *               [0, num_pages) are not visible; a sequence length outside
 *               [0, min(table_width * page_size, 2^30)] counts as 0.  Either is counted
 *               in the error record, by sequence (once or more often), and
 *               never read.
 *   head_dim    1 .. 1024.  Contiguous dims throughout.  Head dims that are
 *               multiples of 16 up to 256, with 16-byte aligned bases and
 *               strides and page and slot strides below 2^31 bytes, take the
 *               tensor-core kernels; the rest a general one.
 *   format, k_scale, v_scale, scales
 *               as kv_gather_fp4 for KV_CACHE_E2M1; forward scales per tensor
 *               (device scalars, NULL: 1) for KV_CACHE_E4M3FN; none for
 *               KV_CACHE_SRC (elements of `dtype`).
 *   work        NULL, or a device workspace of work_bytes (256-byte aligned).
 *               It lets long sequences be split over the GPU and joined; the
 *               more room, the finer (KV_ATTEND_WORK_BYTES is always enough).
 *               Without it each block of query rows of one KV head is one
 *               CTA's work.  Its first KV_ATTEND_HEAD_BYTES are zero before its
 *               first use, and zero again after every call that completes
 *               (zero them after a KV_ERR_CUDA or KV_ERR_WAIT); the rest may
 *               hold anything.
 *               Calls sharing one workspace must not overlap on the GPU.
 * Waits inside the kernels have a limit, far beyond any that ends.  A CTA whose
 * wait ran out leaves rows unwritten, and kv_error_poll returns KV_ERR_WAIT; a
 * call that splits sequences gives NaN for all its rows then.
 * All pointers are device memory, and rejected with KV_ERR_INVALID_ARG where
 * CUDA does not know them.  The result does not depend on the order in which
 * CTAs run, so the same call gives the same bits.  It may differ in rounding
 * with the workspace's size, and with what else the call holds: the kernel, and
 * with it how weights are rounded and where sums are split, is chosen once for the
 * call, from num_seqs, num_q_tokens, table_width and window.
 *
 * Returns KV_OK once enqueued, KV_ERR_INVALID_ARG for a bad argument (NULL
 * pointers, sizes < 1, num_heads not dividing num_q_heads, window or sinks
 * < 0, sm_scale not finite, table_stride < table_width, misaligned scalars or
 * workspace), KV_ERR_UNSUPPORTED for head_dim > 1024, an e2m1 head_dim that is
 * no multiple of 16, or odd 2-byte strides.  num_seqs == 0 or
 * num_q_tokens == 0: KV_OK, nothing launched.
 */
#define KV_ATTEND_WORK_BYTES (64ll << 20)
#define KV_ATTEND_HEAD_BYTES 256
kv_status kv_attend(const void *q, void *out, float *lse, const void *k_cache,
                    const void *v_cache, const int32_t *page_table, int64_t table_stride,
                    int64_t table_width, const int32_t *seq_lens, const int32_t *q_start,
                    int32_t num_seqs, int64_t num_q_tokens, int32_t num_q_heads,
                    int32_t num_heads, int32_t head_dim, kv_src_dtype dtype,
                    const kv_attend_strides *strides, int64_t page_size, int64_t num_pages,
                    kv_cache_format format, const float *k_scale, const float *v_scale,
                    const kv_block_scales *scales, float sm_scale, int64_t window, int64_t sinks,
                    void *work, int64_t work_bytes, kv_error_record *d_err, kv_stream_t stream);

/*
 * A cache of latent rows: one row per token for all query heads, latent_dim
 * dims that attention takes as key and as value, and behind them rope_dim
 * rotated dims that it takes as key only.  The library's 1 x 576 rows (config
 * "odd") are 512 + 64 such dims.  A row lies at
 *     cache + (s / page_size) * cache_page + (s % page_size) * cache_slot
 * for slot s, dims contiguous: KV_CACHE_SRC elements of the source type, or
 * KV_CACHE_E4M3FN bytes with one fp32 scale per slot, scales[s * scale_slot]
 * (a row's value is code * scale).
 */
typedef struct kv_latent_strides {
    int64_t c_token, r_token;        /* bytes between tokens' latent and rotary inputs (dims contiguous) */
    int64_t cache_page, cache_slot;  /* bytes */
    int64_t scale_slot;              /* floats, >= 1 (KV_CACHE_E4M3FN) */
} kv_latent_strides;

/*
 * kv_store_latent -- form the latent rows of new tokens and write them to the
 * cache; rotate the rotary dims of the tokens' queries.
 *
 * For token t:
 *   n = c_t, or with `weight`:  n = fl(fl(c_t * g) * weight),
 *       g = 1 / sqrt(mean(c_t^2) + eps), the mean over the latent dims;
 *   r' = r_t rotated as kv_store_rope does with `rope` (its first rotary_dim
 *       dims, by the token's position);
 *   KV_CACHE_SRC     every element of [n | r'] rounded once to the source type
 *                    (elements that neither step touches keep their bytes);
 *   KV_CACHE_E4M3FN  m = max |[n | r']| (NaN ignored), scale = fl(m / 448),
 *                    codes e4m3fn(fl(x * fl(448 / m))), saturating, where the
 *                    factor may pass fp32's largest number (rows of m below
 *                    2^-119 have the codes of rows 2^64 times as large, and
 *                    subnormal scales); scale and factor are 1 where m is 0.
 * All in fp32; the mean is a sum of fp32 squares (its relative error is below
 * 2^-18 for up to 1,024 dims).
 * rope->q (optional): rotary dims of the queries, [num_tokens, num_q_heads,
 * rope_dim], rotated into rope->q_out, whose token and head strides may be those
 * of whole query rows.
 *
 *   c, r         [num_tokens, latent_dim] and [num_tokens, rope_dim] of
 *                src_dtype; r and rope may be NULL when rope_dim is 0.
 *   weight       NULL, or latent_dim elements of src_dtype.  eps >= 0.
 *   rope         as in kv_store_rope; rotary_dim <= rope_dim.
 * Tokens whose slot or position is out of range: as in kv_store_rope.  Memory
 * kinds as there; weight and scales are device memory.  q_out may be q.
 * latent_dim >= 1, rope_dim >= 0, both together at most 1,024 (else
 * KV_ERR_UNSUPPORTED).  Of tokens that share a slot, codes and scale may be different ones'.
 */
kv_status kv_store_latent(const void *c, const void *r, void *cache, const void *indices,
                          kv_index_dtype index_dtype, int64_t index_stride, int64_t num_tokens,
                          int32_t latent_dim, int32_t rope_dim, kv_src_dtype src_dtype,
                          const kv_latent_strides *strides, int64_t page_size, int64_t size_limit,
                          const void *weight, float eps, const kv_rope *rope,
                          kv_cache_format format, float *scales, kv_error_record *d_err,
                          kv_stream_t stream);

/*
 * kv_gather_latent -- cache rows back: row t of out takes the row_dim dims of
 * slot indices[t], the bytes as they are (KV_CACHE_SRC) or fl16(fl(code *
 * scale)).  strides->c_token is out's token stride; r_token is not used.  An
 * out-of-range slot leaves its row untouched and is counted.  `out` and the
 * slot ids may be page-locked host memory.
 */
kv_status kv_gather_latent(const void *cache, const float *scales, void *out, const void *indices,
                           kv_index_dtype index_dtype, int64_t index_stride, int64_t num_tokens,
                           int32_t row_dim, kv_src_dtype out_dtype, const kv_latent_strides *strides,
                           int64_t page_size, int64_t size_limit, kv_cache_format format,
                           kv_error_record *d_err, kv_stream_t stream);

/* Byte strides of kv_attend_latent, and floats between slots' scales. */
typedef struct kv_attend_latent_strides {
    int64_t q_token, q_head;
    int64_t o_token, o_head;
    int64_t cache_page, cache_slot;
    int64_t scale_slot;
} kv_attend_latent_strides;

/*
 * kv_attend_latent -- causal attention of ragged queries over a paged cache of
 * latent rows.
 *
 * Sequences, queries, pages and positions are kv_attend's.  Every query head
 * reads the same rows k_j of row_dim dims, whose first latent_dim are the
 * values:
 *     s_j = sm_scale * sum_{d < row_dim} q_d k_jd,
 *     out = sum_j exp(s_j) k_j[0 .. latent_dim) / sum_j exp(s_j),
 * over keys j <= the query's position; lse as in kv_attend.  A row that sees no
 * key is 0 with lse -infinity.
 * Statistics and sums are fp32.  16-bit rows are multiplied in their type, e4m3fn
 * codes in fp16 (exact) against queries brought into fp16's range by a power of
 * two per row; a row's scale multiplies its score and its weight in fp32.  The
 * weights meet the values as 16-bit operands (fp16, or bf16 for a bf16 cache),
 * rounded once: up to 2^-9 (bf16) or 2^-12 (fp16) of sum p_j |k_j| / sum p_j
 * beside the output's own rounding.  fp16 weights begin at 2^7 and end at 2^-24.
 *
 *   q            [num_q_tokens, num_q_heads, row_dim] of `dtype`.
 *   out          [num_q_tokens, num_q_heads, latent_dim]; must not overlap q or the cache.
 *   row_dim      1 .. 1024; latent_dim 1 .. row_dim.  Multiples of 16 (row_dim,
 *                up to 576) and 8 (latent_dim, up to 512) with 16-byte aligned
 *                bases and strides, and page and slot strides below 2^31 bytes, take
 *                the tensor-core kernel; the rest a general one.
 *   format       KV_CACHE_SRC or KV_CACHE_E4M3FN (with scales).
 *   sm_scale     of the scores.  Where the keys' up-projection was multiplied into the
 *                queries, the scores are still the products of the head before that: the
 *                scale is 1 / sqrt(its dims, rotary ones included), not 1 / sqrt(row_dim).
 *   work         as in kv_attend (KV_ATTEND_WORK_BYTES is always enough).
 * Page tables, lengths, q_start, waits, errors, determinism and the workspace's
 * head are as in kv_attend.
 */
kv_status kv_attend_latent(const void *q, void *out, float *lse, const void *cache,
                           const float *scales, const int32_t *page_table, int64_t table_stride,
                           int64_t table_width, const int32_t *seq_lens, const int32_t *q_start,
                           int32_t num_seqs, int64_t num_q_tokens, int32_t num_q_heads,
                           int32_t row_dim, int32_t latent_dim, kv_src_dtype dtype,
                           const kv_attend_latent_strides *strides, int64_t page_size,
                           int64_t num_pages, kv_cache_format format, float sm_scale, void *work,
                           int64_t work_bytes, kv_error_record *d_err, kv_stream_t stream);

/*
 * kv_store_noalloc -- kv_store for callers that cannot allocate device memory.
 * The pages have no counterpart; this entry point exists for this library's
 * users only.
 *
 * Some callers cannot call cudaMalloc at the point where they write the KV
 * cache: code running inside an allocator hook (where allocating would
 * re-enter the allocator), a plugin that is handed the tensors but owns no
 * memory pool, or a process whose device memory is entirely reserved by a pool
 * it does not control.  kv_store needs one more device buffer besides the
 * tensors, its error record, so those callers could not use it.
 * kv_store_noalloc takes the same arguments as kv_store except d_err and
 * allocates nothing: the record lives in a 256-byte static device array inside
 * this library (KV_NOALLOC_SCRATCH_BYTES), which every GPU that loads the
 * library holds until the process exits.  The record needs 16 bytes whatever
 * the batch size, so no batch exceeds the array; a build whose record did not
 * fit would return KV_ERR_UNSUPPORTED.
 *
 * Behaviour:
 *  - The first call on a device, with that device current, looks up the
 *    array's device address (cudaGetSymbolAddress); make that first call
 *    before any stream capture on the device.  The address is kept with the
 *    id of the CUDA context it was found in; a call from another context (for
 *    instance after cudaDeviceReset) looks it up again.
 *  - Each call clears the record on `stream`, runs kv_store with it, then
 *    synchronises `stream` and copies the record to *oob_count and
 *    *first_bad_token (host, nullable; -1 when no token was skipped).  It
 *    therefore blocks the host until the write has finished.
 *  - It makes CUDA API calls, so it must not be called from a stream callback
 *    or a host function enqueued with cudaLaunchHostFunc, where CUDA forbids
 *    them.
 *  - Every call shares the one array: calls that overlap on the GPU (from
 *    other host threads or on other streams) race on it and may report each
 *    other's counts.  The cache writes themselves are not affected.
 *  - Calls no cudaMalloc, cudaFree or other allocating routine.
 *
 * Returns KV_OK, KV_ERR_INDEX_OOB when a token was skipped, or the status of
 * kv_store / of a failed CUDA call.
 */
#define KV_NOALLOC_SCRATCH_BYTES 256
kv_status kv_store_noalloc(const void *k, const void *v, void *k_cache, void *v_cache,
                           const void *indices, kv_index_dtype index_dtype, int64_t index_stride,
                           int64_t num_tokens, int32_t num_heads, int32_t head_dim,
                           int32_t elem_bytes, const kv_strides *strides, int64_t size_limit,
                           int32_t num_split, int64_t *oob_count, int64_t *first_bad_token,
                           kv_stream_t stream);

/*
 * kv_error_poll -- synchronise `stream`, read the error record, clear it.
 * (The pages trap inside the kernel on a bad slot; this library reports it
 * here instead.)  Writes the number of skipped tokens and the lowest skipped
 * token (-1 if none) to the optional host outputs.  Returns KV_OK when no
 * token was skipped, KV_ERR_INDEX_OOB when one was, KV_ERR_WAIT when a kernel
 * gave up a wait (whether or not one was), KV_ERR_INVALID_ARG for a
 * NULL or misaligned record, KV_ERR_CUDA if a CUDA call failed (including an
 * earlier asynchronous error surfaced by the synchronisation).
 * Not capturable in a CUDA graph (it synchronises).
 */
kv_status kv_error_poll(kv_error_record *d_err, kv_stream_t stream, int64_t *oob_count,
                        int64_t *first_bad_token);

/* kv_error_snapshot -- copy the record to `dst` asynchronously on `stream`,
 * as it stands once the work before it on the stream has finished.  A small
 * kernel (capturable, chained by programmatic launch), so a captured step can
 * hand its status to the host without a copy-engine transfer: `dst` may be
 * device memory or page-locked host memory (read it after synchronising).
 * The record is not cleared.  Both pointers 8-byte aligned; memory unknown to
 * CUDA is rejected with KV_ERR_INVALID_ARG. */
kv_status kv_error_snapshot(const kv_error_record *d_err, kv_error_record *dst,
                            kv_stream_t stream);

/* kv_error_reset -- zero the record asynchronously on `stream` (capturable). */
kv_status kv_error_reset(kv_error_record *d_err, kv_stream_t stream);

/* kv_launch_floor -- a measurement aid with no counterpart on the pages.
 * Launches an empty kernel sized for num_warps warps of work, with the CTA
 * size, grid and programmatic-launch attributes the write kernels use for
 * that much work, and the same wait for the preceding grid.  It touches no
 * memory.  Timed back to back on a stream, it gives the fixed cost that every
 * launch of this library pays, the floor under a small call such as a decode
 * step (256 tokens of 2048-byte rows run as 1,024 warps).  num_warps in
 * [1, 2^40], else KV_ERR_INVALID_ARG. */
kv_status kv_launch_floor(int64_t num_warps, kv_stream_t stream);

/* Static, NUL-terminated name of a status code. */
const char *kv_status_str(kv_status status);

/* The cudaError_t value of the last failed CUDA call made by this library on
 * the calling thread (0 if none). */
int kv_last_cuda_error(void);

/* KV_ABI_VERSION of the library that was loaded. */
int kv_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FP8_QUANT_GB300_KVSTORE_H */
