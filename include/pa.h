/*
 * pa.h - C ABI of the GB300 PagedAttention step library.
 *
 * One step of a continuous-batching engine's attention layer on one GPU:
 *   1. (optional) rotary embedding of the new Q and K rows,
 *   2. reshape_and_cache: the new K/V rows are written into the shared
 *      paged pool through block_table (in place),
 *   3. causal grouped-query attention of every packed query token over its
 *      sequence's cached context, with optional local window and softcap.
 *
 * The operation is the one specified by "PagedAttention - CUDA Design
 * Document" (onnxruntime 1.29.0 docs, contrib_ops/cuda/paged_attention):
 * section 4 (op contract, input/attribute meaning, in-place cache aliasing),
 * section 4.7 (no host read of device lengths; host values only size
 * launches), section 5.1 (derived write slot), section 8 implementation
 * note P5 (causal bound past + j + 1, window [kv_len - W, kv_len), softcap
 * softcap * tanh(x * scale / softcap), split-KV with log-sum-exp merge),
 * section 9 (-1 block entries are unmapped and masked) and section 15
 * (validation rules); and by "Design: WebGPU PagedAttention" section 3.3
 * (packed tokens delimited by cumulative_sequence_lengths).
 *
 * Conventions for every entry point
 *   - All tensor pointers are DEVICE pointers on the handle's device unless
 *     stated otherwise; all tensors are dense row-major.  fp16 tensors are
 *     passed as void* holding IEEE binary16.  int32 tensors as int32_t*.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default).
 *   - The caller owns every tensor.  key_cache and value_cache are updated
 *     in place (the op's cache outputs alias its cache inputs).  The library
 *     owns only the workspace allocated by pa_create.
 *   - pa_cache_write and pa_forward never allocate, never synchronise and
 *     never copy device data to the host, so they may be captured into a CUDA
 *     graph (device addresses must then stay fixed across replays).
 *   - Host-checkable errors return PA_INVALID_ARGUMENT / PA_NOT_SUPPORTED
 *     before anything is launched; pa_last_error_message() names the
 *     offending argument.  Device-resident values (lengths, block ids) are
 *     not read by the host: invalid ones are skipped by the kernels without
 *     any out-of-bounds access and recorded in a device error word that
 *     pa_check_device_error() returns.
 *
 * Shapes (T = token_count, B = batch, H = num_heads, Hk = kv_num_heads,
 * D = head_size, bs = block_size, NB = num_blocks, MB = max_blocks_per_seq):
 *   query        [T, H*D]          fp16
 *   key, value   [T, Hk*D]         fp16 (new tokens, not yet rotated)
 *   key_cache    [NB, bs, Hk, D]   fp16, value_cache likewise
 *   block_table  [B, MB]           int32; entry i of row b = block holding
 *                                  positions [i*bs, (i+1)*bs) of sequence b,
 *                                  -1 = not mapped (masked; no write)
 *   cumulative_sequence_lengths [B+1] int32, cum[0] = 0, cum[B] = T
 *   past_sequence_lengths       [B]   int32, cached tokens per sequence
 *   cos_cache, sin_cache [P, rotary_dim/2] fp16 (P = max_rotary_positions)
 *   output       [T, H*D]          fp16
 * Token j of sequence b is packed row cum[b] + j and has position
 * past[b] + j.  Query head h uses kv head h / (H / Hk).
 *
 * Quantized cache (section 8): with cache_dtype PA_CACHE_INT8 or
 * PA_CACHE_FP8_E4M3 the pools hold one signed 8-bit code per element,
 * [NB, bs, Hk, D] bytes, with zero point 0: element value = code * scale.
 * k_scale / v_scale are fp32, [1] (PA_QUANT_PER_TENSOR) or [Hk, D]
 * (PA_QUANT_PER_CHANNEL: kv head k's channel c uses scale[k*D + c]).
 * head_sink (section 6) is an optional fp16 [H]: one extra logit per query
 * head that enters the softmax denominator only.  Both arrive through
 * pa_extra_inputs (pa_cache_write_ex / pa_forward_ex).
 *
 * Packed QKV (section 4): with packed_qkv the query argument holds rows
 * [T, (H + 2*Hk)*D] = [Q heads | K heads | V heads] and key / value are NULL.
 * QK-Norm (section 7): with qk_norm every head of Q and K is replaced, before
 * rotary and before K is cached, by
 *   y[c] = fp16((x[c] * r) * w[c]),  r = 1 / sqrt(sum_j x[j]^2 / D + eps),
 * w = q_norm_weight / k_norm_weight ([D] fp16, shared by all heads); the
 * fp32 sum of squares is one running sum over the channels in ascending
 * order (one rounding per square and per add), then IEEE square root and
 * reciprocal, so the cached K is bit-reproducible.
 */
#ifndef PA_H_
#define PA_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define PA_API __attribute__((visibility("default")))
#else
#define PA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef struct pa_handle_s* pa_handle;

typedef enum {
  PA_OK = 0,
  PA_INVALID_ARGUMENT = 1,   /* a host-checkable rule was violated */
  PA_NOT_SUPPORTED = 2,      /* valid op, but not built here (e.g. head_size 80) */
  PA_CUDA_ERROR = 3,         /* a CUDA runtime/driver call failed */
  PA_DEVICE_DATA_ERROR = 4   /* pa_check_device_error found a flagged value */
} pa_status;

/* Bits of the device error word (pa_check_device_error). */
enum {
  PA_DEVERR_CUM = 1,          /* cum[0] != 0, cum not monotone or cum[B] != T */
  PA_DEVERR_BLOCK_ID = 2,     /* block id outside [-1, NB) (access skipped) */
  PA_DEVERR_PAST = 4,         /* past < 0 (sequence skipped) */
  PA_DEVERR_KV_BOUND = 8,     /* past + q_len > kv bound or > MB*bs (sequence skipped) */
  PA_DEVERR_Q_BOUND = 16,     /* q_len > max_query_len_bound (sequence skipped) */
  PA_DEVERR_ROTARY_POS = 32,  /* position >= max_rotary_positions (row left unrotated) */
  PA_DEVERR_TIMEOUT = 64,     /* an internal wait exceeded its limit (kernel gave up; see pa_last_wait_site) */
  PA_DEVERR_SLOT = 128,       /* slot_mapping entry outside [-1, NB*bs) (row not written) */
  PA_DEVERR_ACCEPTED = 256,   /* pa_tree_commit: accepted path not ascending or out of range (sequence skipped) */
  PA_DEVERR_PAGES = 512       /* pa_pages_*: out of free pages, a bad parent, or a page copied twice (row or pair skipped) */
};

/* Cache element types (section 8.2, T_CACHE).  8-bit codes are signed and
 * zero-symmetric; writing a value x stores code = Q(x / scale) with the
 * division in fp32 and Q = round to nearest-even saturated to [-128, 127]
 * (int8) or to +-448 (e4m3fn).
 * PA_CACHE_BF16 selects bfloat16 activations with a bfloat16 cache (section
 * 8.2 registers the kernel for fp16 and bfloat16 activations): query, key,
 * value, both pools, cos_cache / sin_cache, head_sink and the output are
 * then bfloat16 wherever this header says fp16.  Rotary rounds each rotated
 * value to bfloat16 (nearest-even) after the same fp32 arithmetic; the
 * attention contractions take bfloat16 operands (the softmax weights P are
 * rounded to bfloat16 for the P*V contraction) with fp32 accumulation;
 * QK-Norm weights are bfloat16 and its outputs rounded to bfloat16.  The
 * latent layout and pa_forward_no_alloc are fp16 only (PA_NOT_SUPPORTED). */
enum { PA_CACHE_FP16 = 0, PA_CACHE_INT8 = 1, PA_CACHE_FP8_E4M3 = 2, PA_CACHE_BF16 = 3 };

/* Activation types (section 8.2 registers fp16 and bfloat16 activations
 * with every cache type).  PA_ACT_DEFAULT: fp16, or bfloat16 with
 * PA_CACHE_BF16.  PA_ACT_BF16 with an 8-bit cache: query, key, value,
 * cos_cache / sin_cache, head_sink, the QK-Norm weights and the output are
 * bfloat16, transformed (QK-Norm, rotary) with the bfloat16 roundings above;
 * the codes are those of the bfloat16 values (division in fp32).  The
 * attention contractions run on fp16 operands as for fp16 activations (the
 * query is copied as fp16, exact for bfloat16 values in fp16's normal range;
 * |q| beyond 65504 overflows there).  With PA_CACHE_FP16 it is
 * PA_INVALID_ARGUMENT; pa_forward_no_alloc takes PA_ACT_DEFAULT only. */
enum { PA_ACT_DEFAULT = 0, PA_ACT_BF16 = 1 };
/* Cache layout (section 12).  LATENT: one cache key_cache [NB, bs, 1, D] of
 * latent rows (value and value_cache NULL, kv_num_heads 1); every query
 * head attends with its D channels and the output is the weighted sum of
 * the first v_head_size channels of the same rows (absorbed multi-head
 * latent attention); an explicit scale is required.  Built: D = 576,
 * v_head_size = 512, num_heads <= 16 or a multiple of 16, fp16 cache;
 * output [T, H*512].  A sequence with several new tokens (chunked prefill,
 * prefix caching) runs in the same absorbed form, each token attending
 * causally like a one-token decode row (section 12.8). */
enum { PA_LAYOUT_SEPARATE = 0, PA_LAYOUT_LATENT = 1 };
/* Scale granularity (section 8.2, k_quant_type / v_quant_type). */
enum { PA_QUANT_NONE = 0, PA_QUANT_PER_TENSOR = 1, PA_QUANT_PER_CHANNEL = 2 };

/* Static description of a layer, fixed for the handle's lifetime
 * (section 4.5 attributes plus the capacities that size launches, 4.7). */
typedef struct {
  int num_heads;          /* H, > 0, multiple of kv_num_heads */
  int kv_num_heads;       /* Hk, > 0 */
  int head_size;          /* D, multiple of 8; the library runs 64, 128, 256 (576 with the latent layout) */
  int block_size;         /* bs, power of two >= 16 */
  int num_blocks;         /* NB, > 0 */
  int max_blocks_per_seq; /* MB, > 0 (block_table row length) */
  float scale;            /* 0 => 1/sqrt(D) */
  float softcap;          /* 0 => off; > 0 => softcap*tanh(x/softcap) */
  int local_window_size;  /* -1 => off; W >= 1 admits W positions incl. self */
  int do_rotary;          /* 0/1: rotate Q and K before the write */
  int rotary_interleaved; /* 0: pairs (i, i+R/2); 1: pairs (2i, 2i+1) */
  int rotary_dim;         /* R = 2*cos_cache.shape[1]; 0 => D when do_rotary */
  int max_rotary_positions; /* P = cos_cache.shape[0] (rows of the tables) */
  int max_batch;          /* capacity for B across every call on the handle */
  int max_tokens;         /* capacity for T across every call on the handle */
  int max_query_len_bound; /* 0 => max_tokens; upper bound on any q_len */
  int max_kv_len_bound;    /* 0 => MB*bs; upper bound on any past + q_len */
  int cache_dtype;         /* PA_CACHE_*: element type of key_cache / value_cache */
  int k_quant_type;        /* PA_QUANT_*: NONE for 16-bit caches, else PER_TENSOR / PER_CHANNEL */
  int v_quant_type;        /* must equal k_quant_type */
  int packed_qkv;          /* 1: pa_forward's query rows are [Q heads | K heads | V heads], key/value NULL */
  int qk_norm;             /* 1: QK-Norm of Q and K before rotary (q/k_norm_weight required) */
  float qk_norm_epsilon;   /* > 0 (default 1e-6) */
  int kv_cache_layout;     /* PA_LAYOUT_SEPARATE (key_cache + value_cache) or PA_LAYOUT_LATENT */
  int v_head_size;         /* 0 => head_size; != head_size only with PA_LAYOUT_LATENT */
  int rotary_offset;       /* first rotated channel of a head (multiple of 8; latent: v_head_size) */
  int act_dtype;           /* PA_ACT_*: activation type (PA_ACT_BF16 with an 8-bit cache) */
} pa_config;

/* Fills *cfg with the attribute defaults (scale 0, softcap 0, window -1,
 * no rotary, bounds 0, fp16 cache, no packed QKV, no QK-Norm, QK-Norm
 * epsilon 1e-6).  Geometry fields are set to 0 and must be filled. */
PA_API void pa_config_init(pa_config* cfg);

/* Host-only check of a configuration against the validation rules
 * (section 15): H % Hk == 0, D % 8 == 0, bs a power of two >= 16,
 * softcap >= 0, window == -1 or >= 1, rotary_dim even and <= D, positive
 * capacities, quantization NONE exactly for 16-bit caches.  Writes a message
 * naming the field into msg (may be NULL).  Returns PA_INVALID_ARGUMENT or
 * PA_NOT_SUPPORTED on failure.  Not built (PA_NOT_SUPPORTED): 8-bit caches
 * with head_size 64, with k_quant_type != v_quant_type, or with
 * num_heads / kv_num_heads above 16 (8-bit caches run every query row
 * through the decode kernel: a sequence whose q_len * num_heads /
 * kv_num_heads rows exceed one 16-row item runs in chunks of
 * 16 * kv_num_heads / num_heads tokens, section 8.5); a bfloat16 cache
 * with the latent layout.  Touches no GPU. */
PA_API pa_status pa_validate_config(const pa_config* cfg, char* msg, size_t msg_len);

/* Host-only check of one step's arguments (token_count <= max_tokens,
 * batch <= max_batch, required pointers non-NULL (query, key, value and
 * output may be NULL when token_count == 0), rotary tables present iff
 * do_rotary).  query/output may be NULL when checking pa_cache_write
 * (pass for_forward = 0).  Touches no GPU. */
PA_API pa_status pa_check_step(const pa_config* cfg, int for_forward, const void* query,
                        const void* key, const void* value, const void* key_cache,
                        const void* value_cache, const int32_t* block_table,
                        const int32_t* cumulative_sequence_lengths,
                        const int32_t* past_sequence_lengths, int batch,
                        int token_count, const void* cos_cache,
                        const void* sin_cache, const void* output, char* msg,
                        size_t msg_len);

/* Validates cfg, then allocates the device workspace on the current CUDA
 * device (work lists, split-KV partials, rotated-query buffer, error word)
 * sized from the capacities.  May synchronise; never call during capture.
 * On failure *out is NULL and pa_last_error_message(NULL) explains. */
PA_API pa_status pa_create(const pa_config* cfg, pa_handle* out);

/* Steps 1-2 only: rotary on K (if do_rotary) and the paged write of K and V
 * for every new token.  Slot = block_table[b][pos/bs]*bs + pos%bs; a -1
 * entry writes nothing.  Bit-exact: without rotary the rows are copied;
 * with rotary each pair is y1 = x1*c - x2*s, y2 = x2*c + x1*s in fp32 with
 * one rounding per operation, then rounded to fp16. */
PA_API pa_status pa_cache_write(pa_handle h, const void* key, const void* value,
                         void* key_cache, void* value_cache,
                         const int32_t* block_table,
                         const int32_t* cumulative_sequence_lengths,
                         const int32_t* past_sequence_lengths, int batch,
                         int token_count, const void* cos_cache,
                         const void* sin_cache, void* stream);

/* The whole step: rotary on Q and K (if do_rotary), the paged cache write,
 * then attention for every packed query row into output.  Row (t, h) of
 * sequence b attends to positions p in [lo, past_b + j + 1) with
 * lo = max(0, past_b + j + 1 - W) under a window, skipping positions whose
 * block entry is -1; x = scale * <q, k_p>, optionally softcapped; output is
 * the softmax-weighted sum of v_p (0 when no position is admitted).
 * token_count == 0 returns PA_OK and launches nothing. */
PA_API pa_status pa_forward(pa_handle h, const void* query, const void* key,
                     const void* value, void* key_cache, void* value_cache,
                     const int32_t* block_table,
                     const int32_t* cumulative_sequence_lengths,
                     const int32_t* past_sequence_lengths, int batch,
                     int token_count, const void* cos_cache,
                     const void* sin_cache, void* output, void* stream);

/* Optional inputs of the op contract (section 4, inputs 11, 14, 15).  Any
 * pointer may be NULL where its feature is off. */
typedef struct {
  const void* head_sink;  /* [H] fp16, device; NULL = no sink */
  const float* k_scale;   /* device fp32, [1] or [Hk*D]; required iff the cache is 8-bit */
  const float* v_scale;   /* likewise for value_cache */
  const int32_t* slot_mapping; /* [T] int32, device; NULL = derive the write slot from block_table */
  const void* q_norm_weight;   /* [D] fp16, device; required iff qk_norm (with k_norm_weight) */
  const void* k_norm_weight;   /* [D] fp16, device */
} pa_extra_inputs;

/* pa_cache_write with the optional inputs (extra may be NULL).  With an
 * 8-bit cache the written rows are quantized (after rotary) under
 * k_scale / v_scale as stated at PA_CACHE_INT8; bit-exact.
 * slot_mapping (section 5.2) is authoritative for the write: packed row t
 * goes to flat slot slot_mapping[t] of the pool viewed as [NB*bs, Hk, D];
 * -1 writes nothing (the row's query still attends); values outside
 * [-1, NB*bs) write nothing and set PA_DEVERR_SLOT.  block_table still
 * defines what every sequence reads (positions [i*bs, (i+1)*bs) of row b),
 * so a runtime can recycle blocks, e.g. a ring of ceil(W/bs)+1 blocks per
 * sequence under a local window W with -1 entries below the window
 * (section 9.3). */
PA_API pa_status pa_cache_write_ex(pa_handle h, const void* key, const void* value,
                                   void* key_cache, void* value_cache,
                                   const int32_t* block_table,
                                   const int32_t* cumulative_sequence_lengths,
                                   const int32_t* past_sequence_lengths, int batch,
                                   int token_count, const void* cos_cache,
                                   const void* sin_cache, const pa_extra_inputs* extra,
                                   void* stream);

/* pa_forward with the optional inputs (extra may be NULL).  8-bit caches
 * are read at their stored width: a per-tensor K scale multiplies the
 * softmax scale, per-channel K scales are folded into the query
 * (q * k_scale[c], rounded to fp16), and the V scale multiplies the output
 * (section 8.5 phase 3).  head_sink s_h adds exp(s_h - m) to the softmax
 * denominator of every row of head h, m = max(s_h, max logit) (section
 * 6.1); a row with no admitted key still outputs 0. */
PA_API pa_status pa_forward_ex(pa_handle h, const void* query, const void* key,
                               const void* value, void* key_cache, void* value_cache,
                               const int32_t* block_table,
                               const int32_t* cumulative_sequence_lengths,
                               const int32_t* past_sequence_lengths, int batch,
                               int token_count, const void* cos_cache,
                               const void* sin_cache, const pa_extra_inputs* extra,
                               void* output, void* stream);

/* Synchronises the stream of the handle's last call, reads and clears the
 * device error word into *code (0 = clean).  Returns PA_DEVICE_DATA_ERROR
 * when *code != 0.  Not capturable.  With PA_DEVERR_TIMEOUT set, the message
 * (pa_last_error_message) and pa_last_wait_site name the wait that gave up. */
PA_API pa_status pa_check_device_error(pa_handle h, int* code);

/* Wait sites.  Every bounded wait inside the library's kernels has an id
 * (kernel << 8) | index; the first wait of a step that gives up records
 * it beside the error word.  Kernel parts of the id: */
enum {
  PA_SITE_DECODE = 1 << 8,
  PA_SITE_COMBINE = 2 << 8,        /* index 1: the PA_OPT_WAIT_PROBE wait */
  PA_SITE_PREFILL = 3 << 8,        /* one-tile prefill (head_size 256) */
  PA_SITE_PREFILL_PAIR = 4 << 8,   /* two-tile prefill (head_size 64, 128) */
  PA_SITE_LATENT = 5 << 8,         /* latent decode, mma.sync */
  PA_SITE_LATENT_TC = 6 << 8,      /* latent decode, tcgen05 */
  PA_SITE_TREE = 7 << 8,           /* tree attention */
  PA_SITE_Q4 = 8 << 8              /* attention over 4-bit pools */
};
/* The wait-site id read (and cleared) by the last pa_check_device_error on
 * h; 0 when no wait gave up. */
PA_API int pa_last_wait_site(pa_handle h);

/* Message of the last failure on h (or of the last pa_create / validation
 * failure on this thread when h is NULL).  Never NULL. */
PA_API const char* pa_last_error_message(pa_handle h);

/* Frees the workspace.  NULL is accepted. */
PA_API pa_status pa_destroy(pa_handle h);

/* The whole step (as pa_forward) for callers that cannot allocate device
 * memory: code running inside CUDA stream capture, under a memory pool
 * they do not own, in an allocation-free serving loop, or that simply has
 * no handle.  The design pages have no counterpart to this call.
 *
 * It needs no pa_create: cfg is passed on every call, and every scratch
 * buffer (work lists, split-KV partials, the rotated-query buffer, the
 * device error word) lives in one file-scope device array of 64 MiB that
 * each GPU loading this library holds until the process exits.  The call
 * makes no cudaMalloc/cudaFree and no other allocation; the caller still
 * passes every input and the output.  Capacities (max_batch, max_tokens,
 * head counts, head_size, do_rotary) whose scratch would exceed 64 MiB are
 * rejected with PA_INVALID_ARGUMENT and a message giving the size needed.
 *
 * device_error: optional caller-owned device int32 that receives the
 * PA_DEVERR_* bits (OR-ed; the caller clears it).  When NULL the bits go
 * to a word inside the shared scratch, cleared at the start of each call,
 * that the caller cannot read (so is the wait-site id of a timeout).
 *
 * It runs separate fp16 K/V caches without head_sink; an 8-bit or bfloat16
 * cache_dtype, packed_qkv, qk_norm or kv_cache_layout PA_LAYOUT_LATENT
 * returns PA_NOT_SUPPORTED (pa_forward_ex takes all of them and the sink).
 *
 * The first call on a device does a one-time set-up with that device
 * current (looks up the array's device address with cudaGetSymbolAddress,
 * sets the kernels' shared-memory attributes); make that first call before
 * any stream capture.  All calls share the one scratch array, which keeps
 * the last call's contents: calls that can overlap on the GPU (different
 * streams, or concurrent graphs) race on it and must be serialised by the
 * caller. */
PA_API pa_status pa_forward_no_alloc(const pa_config* cfg, const void* query, const void* key,
                                     const void* value, void* key_cache, void* value_cache,
                                     const int32_t* block_table,
                                     const int32_t* cumulative_sequence_lengths,
                                     const int32_t* past_sequence_lengths, int batch,
                                     int token_count, const void* cos_cache,
                                     const void* sin_cache, void* output,
                                     int32_t* device_error, void* stream);

/* ---- tuning and measurement hooks (set outside capture) ---- */
enum {
  PA_OPT_SPLIT_KEYS = 1,      /* > 0: fixed keys per decode split (multiple of 64); 0 = auto */
  PA_OPT_NO_WINDOW_PRUNE = 2, /* 1: walk the whole context and mask instead of pruning */
  PA_OPT_KERNEL_TIMING = 3,   /* 1: record CUDA events around each kernel of pa_forward */
  PA_OPT_DECODE_MAX_ROWS = 4, /* route a sequence to the decode kernel iff q_len*G <= value (0 = never; at most and by
                                 default the rows of a decode item: 8 when G <= 8, else 16) */
  PA_OPT_DECODE_ITEMS_PER_CTA = 5, /* target decode work items per decode CTA when splits are sized automatically:
                                      1..32, or 0 (default) = per step, 1 when the step's sequences x kv heads
                                      (latent: x work units per sequence) fill the decode grid, else 2 */
  PA_OPT_LATENT_TCGEN05 = 6,  /* latent layout: 1 (the default when the query heads are a multiple of 128)
                                 runs the tcgen05 latent kernel (units of 128 heads x half the value
                                 channels), 0 the mma.sync kernel (items of 32 heads, any head count);
                                 1 on other handles is PA_NOT_SUPPORTED */
  PA_OPT_PREFILL_SMS = 7,     /* steps with prompts and decode rows: the prefill kernel runs on P SMs and the
                                 decode kernel beside it on the rest; 0 (default) = P from the step's own work
                                 (cost model), -1 = no split (every prefill CTA works, the decode kernel
                                 fills SMs as they free), > 0 = P fixed (at most SMs - 1) */
  PA_OPT_WAIT_PROBE = 8       /* 1: the combine kernel also runs a bounded wait (2 ms) on a flag nothing sets,
                                 so that the step ends with PA_DEVERR_TIMEOUT at site PA_SITE_COMBINE | 1
                                 (a check of the timeout path; the step's outputs are unaffected) */
};
PA_API pa_status pa_set_option(pa_handle h, int option, int value);

/* Kernel stages of a step, for pa_kernel_time_ms.  In pa_forward the work
 * list and the cache write run as one launch (the prologue), timed as
 * PA_STAGE_WORKLIST; PA_STAGE_CACHE_WRITE times pa_cache_write. */
enum {
  PA_STAGE_WORKLIST = 0,
  PA_STAGE_CACHE_WRITE = 1,
  PA_STAGE_DECODE = 2,
  PA_STAGE_PREFILL = 3,
  PA_STAGE_COMBINE = 4,
  PA_NUM_STAGES = 5
};
/* With PA_OPT_KERNEL_TIMING on: synchronises, then returns in *ms the time
 * between the events recorded on the launch stream around that stage's
 * kernel in the last pa_forward (-1 when it did not launch). */
PA_API pa_status pa_kernel_time_ms(pa_handle h, int stage, float* ms);

/* Number of kernels the last pa_forward / pa_cache_write launched. */
PA_API int pa_last_launch_count(pa_handle h);

/* What the device work list of the last pa_forward on h decided (an
 * inspection hook for tests and tuning; synchronises, not capturable):
 * counts[PA_STEP_COUNTS] receives decode work items (sequence, split),
 * prefill tiles, packed rows merged by the combine kernel, keys per decode
 * split, prefill CTAs kept and decode CTAs kept (with the SM split of a
 * mixed step their sum is at most the SM count times the decode CTAs per
 * SM; without it they are the launched grids). */
enum { PA_STEP_COUNTS = 6 };
PA_API pa_status pa_last_step_counts(pa_handle h, int32_t* counts);

/* ---- speculative decoding: trees of drafted tokens ----
 *
 * The new tokens of a sequence may be a tree of drafted tokens instead of a
 * run.  Draft token j of sequence b (packed row t = cum[b] + j, parents
 * before children) occupies cache slot past[b] + j until the step is decided,
 * but stands at its own position (past[b] + its depth, as a rule) and attends
 * to the cached context and to its own ancestors.  The calls, in order:
 *   pa_tree_write      Q and K rotated at explicit positions, Q to a dense
 *                      copy, K and V to slots past[b] + j of the paged pool
 *   pa_tree_attention  attention under a mask over the draft tokens
 *   pa_tree_commit     the accepted path's rows moved to the front of the
 *                      draft slots, in every layer's pools
 * pa_rotary is the same rotation on plain rows, and its gradient.
 *
 * Padding: rows at and behind cum[batch] (cum[batch] <= token_count) are
 * not written and what they hold does not matter, so a captured step may be
 * sized for more tokens than it holds. */

/* Element types of pa_rotary. */
enum { PA_ROTARY_FP16 = 0, PA_ROTARY_BF16 = 1, PA_ROTARY_FP32 = 2 };

/* Frequency scalings for contexts longer than the trained one (R =
 * rotary_dim, f_i = base^(-2i/R) radians per position for pair i, s =
 * factor, L = original_positions):
 *   NONE           f_i
 *   LINEAR         f_i / s
 *   BASE           (base * s^(R/(R-2)))^(-2i/R)
 *   BY_PARTS       f_i/s * r_i + f_i * (1 - r_i), r_i = clamp((i - lo)/(hi - lo), 0, 1),
 *                  lo = max(floor(at(high)), 0), hi = min(ceil(at(low)), R - 1),
 *                  at(turns) = R ln(L/(2 pi turns)) / (2 ln base);
 *                  attention factor 0.1 ln(s) + 1
 *   BY_WAVELENGTH  f_i/s * (1 - k_i) + f_i * k_i, k_i = clamp((L f_i/(2 pi) - low)/(high - low), 0, 1)
 * low < high are turns over the L original positions. */
enum {
  PA_ROTARY_SCALE_NONE = 0,
  PA_ROTARY_SCALE_LINEAR = 1,
  PA_ROTARY_SCALE_BASE = 2,
  PA_ROTARY_SCALE_BY_PARTS = 3,
  PA_ROTARY_SCALE_BY_WAVELENGTH = 4
};
typedef struct {
  int type;                  /* PA_ROTARY_SCALE_* */
  double base;               /* > 1 */
  double factor;             /* s >= 1; read unless NONE */
  double original_positions; /* L > 0; BY_PARTS and BY_WAVELENGTH */
  double low, high;          /* 0 < low < high; BY_PARTS and BY_WAVELENGTH */
} pa_rotary_scaling;

/* Host only: steps[i] = the frequency of pair i as 2^-64 turns per position,
 * round(f_i / (2 pi) * 2^64) mod 2^64, i < rotary_dim / 2.  The phase of
 * position p is then (p * steps[i]) mod 2^64, exact in wrapping 64-bit
 * arithmetic however far p is (also negative).  *attention_factor (may be
 * NULL) receives the factor on cos and sin (1 except BY_PARTS).  The caller
 * copies the steps to the device; own frequencies may be given the same way. */
PA_API pa_status pa_rotary_steps(const pa_rotary_scaling* scaling, int rotary_dim, uint64_t* steps,
                                 float* attention_factor);

/* Row geometry of a rotation. */
typedef struct {
  int head_size;          /* D, multiple of 8, at most 512 */
  int rotary_dim;         /* R, multiple of 16; 0 => D */
  int rotary_offset;      /* first rotated channel, multiple of 8 */
  int interleaved;        /* 0: pairs (i, i+R/2); 1: pairs (2i, 2i+1) */
  int dtype;              /* PA_ROTARY_* */
  float attention_factor; /* m, finite; 1 by default */
  int conjugate;          /* 1: rotate by -angle; with the same m this is the gradient of the rotation
                             (dx from dy), with 1/m it is its inverse */
} pa_rotary_config;
/* Zeroes *rc, attention_factor 1. */
PA_API void pa_rotary_config_init(pa_rotary_config* rc);

/* Rotates token_count rows of Q and K at positions[t] (int32, device, any
 * value): per pair, with a = 2 pi frac(positions[t] * steps[i] / 2^64),
 *   y1 = m (x1 cos a - x2 sin a),  y2 = m (x2 cos a + x1 sin a)
 * in fp32, rounded once to the type; the other channels are copied.
 * Row t of a tensor starts at t * stride elements (a multiple of 8, at least
 * heads * D; 0 => heads * D; one row has no stride), so slices of packed rows
 * are taken and written in place.  query_out == query with equal strides
 * rotates in place; an output that overlaps its input in any other way is
 * refused, and so are outputs that overlap each other, the other input,
 * positions or steps.
 * Overlap is decided by whole ranges of rows, save that two slices of one row
 * layout (equal strides, disjoint columns) do not overlap.  num_heads or
 * kv_num_heads 0 leaves that tensor out (at most 4096 of each).  Runs on the
 * current device; keeps nothing, so calls may overlap. */
PA_API pa_status pa_rotary(const pa_rotary_config* rc, const uint64_t* steps, const int32_t* positions,
                           int token_count, int num_heads, const void* query, int64_t query_stride,
                           void* query_out, int64_t query_out_stride, int kv_num_heads, const void* key,
                           int64_t key_stride, void* key_out, int64_t key_out_stride, void* stream);

typedef struct pa_tree_handle_s* pa_tree_handle;

/* A layer's handle for trees of at most max_draft_tokens (1..256) drafted
 * tokens per sequence.  cfg is the layer's pa_config; read are the heads,
 * head_size, paging, scale, softcap, local_window_size, max_batch,
 * max_tokens, max_kv_len_bound and cache_dtype (PA_CACHE_FP16 or
 * PA_CACHE_BF16, the activations' type too).  Its rotary fields are not read
 * here (positions are explicit; pa_tree_write takes a pa_rotary_config).
 * PA_NOT_SUPPORTED: 8-bit caches, the latent layout, packed_qkv, qk_norm,
 * more than 4096 heads.  Allocates the workspace (split-KV partials, error
 * word) on the current device; other calls run there whatever is current.
 * Flagged (PA_DEVERR_KV_BOUND): a sequence of 2^26 key tiles (128 keys by up
 * to 256 query rows of a kv head; 64 by 128 at head_size 256) or more, and a
 * batch of 2^31.
 * One handle's pa_tree_attention calls share that workspace: calls (and
 * replays of graphs captured from them) on one handle must not overlap on the
 * GPU; use a handle per stream.  pa_tree_write and pa_tree_commit do not use it. */
PA_API pa_status pa_tree_create(const pa_config* cfg, int max_draft_tokens, pa_tree_handle* out);
PA_API pa_status pa_tree_destroy(pa_tree_handle h);

/* pa_rotary on Q and K (rc->head_size and dtype must be the handle's), then
 * K and V to slots past[b] + j of the paged pools through block_table (a -1
 * entry writes nothing).  query_out [T, H*D] dense; query_out may be query
 * when query_stride is H*D.  V rows are copied bit for bit.  positions [T].
 * query_out and the pools must not overlap any other input. */
PA_API pa_status pa_tree_write(pa_tree_handle h, const pa_rotary_config* rc, const uint64_t* steps,
                               const int32_t* positions, const void* query, int64_t query_stride,
                               const void* key, int64_t key_stride, const void* value, int64_t value_stride,
                               void* query_out, void* key_cache, void* value_cache, const int32_t* block_table,
                               const int32_t* cumulative_sequence_lengths, const int32_t* past_sequence_lengths,
                               int batch, int token_count, void* stream);

/* Optional inputs of pa_tree_attention; any pointer may be NULL. */
typedef struct {
  const int32_t* positions;     /* [T]; NULL => past[b] + j.  Used by the window and the distance bias */
  const uint32_t* tree_mask;    /* [T, ceil(max_draft_tokens/32)]: bit i%32 of word i/32 of row t admits draft
                                   token i of the same sequence; bits at and above its length are ignored, no bit
                                   is implied.  NULL => causal (i <= j) */
  const float* distance_slopes; /* [H]: adds slope_h * (kpos - qpos) to the scores, after softcap */
  const void* head_sink;        /* [H], the cache's type: one extra logit in the denominator */
} pa_tree_inputs;

/* Attention of every packed query row over its sequence's cache (the draft
 * rows already written).  Row (t, h) admits every context slot p < past[b]
 * (at position p; -1 pages are masked) and draft token i under the mask (at
 * positions[cum[b] + i]); with local_window_size W only keys at positions
 * > max(positions[t], past[b]) - W.  x = scale <q, k>, softcapped, plus the
 * bias (positions of a sequence's keys and rows within 2^31 of one another);
 * output = sum softmax(x) v, 0 when nothing is admitted.  A key that a row
 * does not admit never reaches that row, whatever its K and V hold (under a
 * window this holds for rows at positions below past[b] + max_draft_tokens;
 * a row further on needs finite V at its window's edge).  A score that is
 * NaN or +inf makes its row NaN, and a non-finite V of an admitted key that
 * channel of the row.  query, output [T, H*D]; output must not overlap the
 * inputs.  P is rounded to the 16-bit type for the P*V contraction; scores,
 * sums and the output accumulate in fp32 (a distance bias is held to 2^-22 of
 * |slope| (128 + |kpos - qpos|)). */
PA_API pa_status pa_tree_attention(pa_tree_handle h, const void* query, const void* key_cache,
                                   const void* value_cache, const int32_t* block_table,
                                   const int32_t* cumulative_sequence_lengths,
                                   const int32_t* past_sequence_lengths, int batch, int token_count,
                                   const pa_tree_inputs* inputs, void* output, void* stream);

/* For every sequence b and layer l: slot past[b] + i receives the K and V rows
 * of slot past[b] + accepted[b * max_accepted + i], i < accepted_count[b].
 * accepted rows are strictly ascending draft indexes below max_draft_tokens
 * (a path in packed order), with max_accepted <= max_draft_tokens.
 * key_caches and value_caches are HOST arrays of num_layers device pointers
 * to pools of the handle's geometry, none overlapping another.  new_past [batch] (may be NULL, must
 * not overlap any input) receives past[b] + accepted_count[b].  A sequence with a
 * bad path or length is left as it was (new_past = past) and flagged; a -1
 * page moves nothing. */
PA_API pa_status pa_tree_commit(pa_tree_handle h, void* const* key_caches, void* const* value_caches,
                                int num_layers, const int32_t* block_table,
                                const int32_t* past_sequence_lengths, const int32_t* accepted,
                                const int32_t* accepted_count, int max_accepted, int batch, int32_t* new_past,
                                void* stream);

/* Synchronises the handle's device, reads and clears the handle's error word
 * (PA_DEVERR_*).  Not capturable. */
PA_API pa_status pa_tree_check_device_error(pa_tree_handle h, int* code);
/* Message of the last failure on h (NULL: on this thread). */
PA_API const char* pa_tree_last_error_message(pa_tree_handle h);

/* ---- pools held in 4 bits ----
 *
 * A cache of 9/32 of the bytes of fp16.  key_cache and value_cache are uint8
 * [NB, Hk, PB], PB = bs * (D/2 + D/16): a page's share of one kv head is one
 * run, the codes of its bs rows (D/2 bytes each), then fp16 scales
 * [D/32, bs].  32 consecutive channels of a row share a scale.  Channel c of
 * row r of the page (j = c / 32, t = c / 8 % 4, i = c % 8): its code is
 * nibble i % 2 * 4 + i / 2 of the little-endian 32-bit word
 * (t ^ (r / 4 % 4)) * (D/32) + j of the row, and its value
 * (code - 8) * scale[j][r].  (The order of the words is the order in which
 * the attention kernels' lanes take them from shared memory.)
 * Pages are copied, forked and compacted like any other's: Hk * PB bytes.
 *
 * A sequence's new rows go to slots past[b] + j through block_table, as in
 * pa_cache_write (-1 writes nothing).  Rows at and behind cum[batch]
 * (cum[batch] <= token_count) are padding: neither read into the pools nor
 * written.  A sequence with a bad length (one that ends behind token_count
 * too) is flagged and left out, its rows as they were. */

/* PB for a block_size (a power of two >= 16) and head_size (64, 128, 256); 0 for others. */
PA_API int64_t pa_q4_page_bytes(int block_size, int head_size);

typedef struct pa_q4_handle_s* pa_q4_handle;

/* A layer's handle.  cfg is the layer's pa_config; read are the heads,
 * head_size, paging, scale, softcap, local_window_size, max_batch, max_tokens,
 * max_kv_len_bound and cache_dtype, which here names the activations' type
 * (PA_CACHE_FP16 or PA_CACHE_BF16).  Its rotary fields are not read: pa_rotary
 * rotates Q and K first.  first_tokens >= 0: under a window, positions below
 * it stay visible.  PA_NOT_SUPPORTED: 8-bit cache_dtypes, the latent layout,
 * packed_qkv, qk_norm, more than 4096 heads.  Allocates the workspace on the current device; other calls run
 * there whatever is current.
 * One handle's pa_q4_attention calls share that workspace: calls (and replays
 * of graphs captured from them) on one handle must not overlap on the GPU;
 * use a handle per stream.  pa_q4_write and pa_q4_read do not use it. */
PA_API pa_status pa_q4_create(const pa_config* cfg, int first_tokens, pa_q4_handle* out);
PA_API pa_status pa_q4_destroy(pa_q4_handle h);

/* Quantizes the rows of key and value [T, Hk*D] (row t at t * stride
 * elements, a multiple of 8; 0 => Hk*D; one row has no stride) into the
 * pools.  Per group of 32 channels, a = max |x|:
 *   scale = fp16(min(a / 7, 65504)), code = clamp(rint(x / scale), -8, 7)
 * with IEEE divisions in 32 bits and rint to nearest even; scale 0 stores
 * zeros, a group with a NaN or an infinity stores NaN as its scale and zero
 * codes.  The same bits on every run.  The pools must not overlap any input. */
PA_API pa_status pa_q4_write(pa_q4_handle h, const void* key, int64_t key_stride, const void* value,
                             int64_t value_stride, void* key_cache, void* value_cache, const int32_t* block_table,
                             const int32_t* cumulative_sequence_lengths, const int32_t* past_sequence_lengths,
                             int batch, int token_count, void* stream);

/* The values held in slots past[b] + j, to rows of key_out and value_out
 * (strides as in pa_q4_write): (code - 8) * scale rounded once to the
 * activations' type; a -1 page reads as zeros.  The outputs must not overlap
 * each other or any input. */
PA_API pa_status pa_q4_read(pa_q4_handle h, const void* key_cache, const void* value_cache,
                            const int32_t* block_table, const int32_t* cumulative_sequence_lengths,
                            const int32_t* past_sequence_lengths, int batch, int token_count, void* key_out,
                            int64_t key_out_stride, void* value_out, int64_t value_out_stride, void* stream);

/* Causal attention of every packed query row over its sequence's pages (the
 * new rows already written).  Row (t, h) at position pos = past[b] + j admits
 * the mapped positions p <= pos; with local_window_size W those with
 * p > pos - W or p < first_tokens.  x = scale <q, k>, softcapped (off by at
 * most 2^-20 of the cap); output =
 * sum softmax(x) v, 0 when nothing is admitted; head_sink [H] (activations'
 * type, may be NULL) adds exp(sink_h) to the denominator.  A key that a row
 * does not admit never reaches that row, whatever its slot holds; an admitted
 * slot of a NaN scale makes the row NaN (its K) or those channels (its V).
 * query and output [T, H*D] dense; output must not overlap the inputs.
 * Scores, sums and the output accumulate in fp32.  A weight times V's scale is
 * rounded to fp16 once.  Sequences of many rows (new tokens x H / Hk) are
 * computed in another way at head_size 64 and 128: an eighth of each value of K
 * and V is rounded to fp16 (values below 2^-11 thus to multiples of 2^-21) and
 * so are the weights, once where they are at least 2^-19 of the largest, and a
 * slot of V with a NaN scale makes the whole row NaN.  Those are sequences of
 * more than 32 rows, 48 in a call with at most 28 batch rows (its token_count x
 * H / Hk), in calls with more tokens than batch or H / Hk > 8; in other calls
 * (single tokens, as a rule) no sequence is, however long. */
PA_API pa_status pa_q4_attention(pa_q4_handle h, const void* query, const void* key_cache, const void* value_cache,
                                 const int32_t* block_table, const int32_t* cumulative_sequence_lengths,
                                 const int32_t* past_sequence_lengths, int batch, int token_count,
                                 const void* head_sink, void* output, void* stream);

/* Synchronises the handle's device, reads and clears the handle's error word
 * (PA_DEVERR_*).  Not capturable. */
PA_API pa_status pa_q4_check_device_error(pa_q4_handle h, int* code);
/* Message of the last failure on h (NULL: on this thread). */
PA_API const char* pa_q4_last_error_message(pa_q4_handle h);

/* ---- the pages of a cache ----
 *
 * What an engine does with pages between steps, on the device: no length is
 * read by the host, so the calls can be captured with the steps around them.
 * A pool is num_blocks pages of page_bytes each (K and V of every layer, of
 * any cache type: a page of a 16-bit pool has bs*Hk*D*2 bytes).  ref_count
 * [NB] says how many block-table entries refer to a page; 0 = free.  Fresh
 * pages are the lowest free ones, handed out in row order, so results do not
 * depend on timing; pages released by a call are free from the next call on.
 * Tables are int32 [rows, max_blocks_per_seq], -1 = no page (an id outside
 * [-1, NB) counts as -1 and is flagged).  pools is a HOST array of num_pools
 * device pointers (none overlapping another); 0 pools moves no bytes.
 * Calls on one handle share its workspace and must not overlap on the GPU
 * (replays of captured ones too). */
typedef struct {
  int block_size;         /* positions of a page, 1..2^20 */
  int num_blocks;         /* NB, 1..2^20 */
  int max_blocks_per_seq; /* entries of a row, at most 2^30 positions */
  int max_rows;           /* most rows of a table, 1..2^20 */
  int64_t page_bytes;     /* bytes of a page in one pool, a multiple of 16, at most 2^32 */
} pa_pages_config;

typedef struct pa_pages_handle_s* pa_pages_handle;
PA_API pa_status pa_pages_create(const pa_pages_config* cfg, pa_pages_handle* out);
PA_API pa_status pa_pages_destroy(pa_pages_handle h);

/* In every pool page dst[i] receives page src[i], i < count <= NB (int32,
 * device).  A -1 on either side leaves the pair out.  Pairs that name one
 * destination are all left out and flagged (PA_DEVERR_PAGES), and so is a pair
 * whose source is any pair's destination. */
PA_API pa_status pa_pages_copy(pa_pages_handle h, void* const* pools, int num_pools, const int32_t* src,
                               const int32_t* dst, int count, void* stream);

/* Rows that take the place of rows: new row i continues row parent[i]
 * (-1: an empty row), so one call forks, reorders and frees sequences.  New
 * row i has the pages of its parent's first lengths[parent] positions; where
 * the last of them is partly filled, the parent's first child keeps it and
 * every other child gets a copy in a fresh page.  new_ref_count = ref_count
 * less the entries of block_table plus those of new_block_table (ref_count
 * itself is allowed for it).  A child that finds no free page is left empty
 * and flagged (PA_DEVERR_PAGES), a parent with a bad length has empty
 * children.  Outputs must not overlap inputs or one another otherwise. */
PA_API pa_status pa_pages_fork(pa_pages_handle h, void* const* pools, int num_pools, const int32_t* block_table,
                               const int32_t* lengths, int rows, const int32_t* parent, int new_rows,
                               const int32_t* ref_count, int32_t* new_block_table, int32_t* new_lengths,
                               int32_t* new_ref_count, void* stream);

/* Row r, of lengths[r] positions, becomes one of lengths[r] + delta[r], in
 * place: missing pages of the new positions are taken from the free ones,
 * and entries behind the last position give theirs back (delta = -length frees
 * the row).  A page of new positions that other entries refer to before the
 * call (a reference count above 1) is replaced by a fresh one, which receives
 * its bytes where positions below lengths[r] lie in it too.  An entry without
 * a page that holds a position below lengths[r] stays as it is.  A row whose
 * pages are not all to be had is left as it was and flagged (PA_DEVERR_PAGES),
 * and so are later rows that need any; so is a row with a bad length, old or
 * new (PA_DEVERR_PAST, PA_DEVERR_KV_BOUND).
 * new_lengths (lengths itself is allowed) receives the lengths that hold. */
PA_API pa_status pa_pages_resize(pa_pages_handle h, void* const* pools, int num_pools, int32_t* block_table,
                                 const int32_t* lengths, const int32_t* delta, int rows, int32_t* new_lengths,
                                 int32_t* ref_count, void* stream);

/* Moves pages so that those in use are [0, n): the i-th used page at or above
 * n goes to the i-th free one below it, in every pool, and table and counts
 * follow (both may be written in place).  pages_in_use [1] receives n. */
PA_API pa_status pa_pages_compact(pa_pages_handle h, void* const* pools, int num_pools, const int32_t* block_table,
                                  int rows, const int32_t* ref_count, int32_t* new_block_table,
                                  int32_t* new_ref_count, int32_t* pages_in_use, void* stream);

/* As pa_q4_check_device_error and pa_q4_last_error_message. */
PA_API pa_status pa_pages_check_device_error(pa_pages_handle h, int* code);
PA_API const char* pa_pages_last_error_message(pa_pages_handle h);

#ifdef __cplusplus
}
#endif
#endif /* PA_H_ */
