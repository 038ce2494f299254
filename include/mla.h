/*
 * mla.h -- C ABI of libmla.so: absorbed Multi-head Latent Attention (MLA)
 * decode on NVIDIA B200 (sm_100a).
 *
 * The method (DeepSeek-V3 MLA, decode step, absorbed order):
 *   - per token and layer the cache keeps only a latent c_KV (d_c = 512) and a
 *     decoupled RoPE key k_R (d_r = 64), 576 numbers
 *     (wq-win.github.io/llm/092-deepseekv3.html, section 二 "MLA：缓存压缩后的历史";
 *      ailearn.mscapital.top/deepseek-v3.html, MLA paragraph after the
 *      configuration table);
 *   - each head's content query is folded through W_UK into latent space and
 *     dotted with every cached c_KV; the RoPE score q_R . k_R is added
 *     separately (092 page, section 二 "缓存压缩也可以做一个代数检查":
 *      q^T (U c) = (U^T q)^T c; m.lsln.cn/news/222502 sections 2.2 and 2.3);
 *   - softmax over the whole history, aggregate sum_j p_j c_KV,j in latent
 *     space, then map through W_UV to the per-head output
 *     (ailearn.mscapital.top/deepseek-v3.html, MLA "状态传导图" panel).
 *
 * Conventions shared by every entry point
 *   - All tensor pointers are DEVICE pointers unless stated otherwise; the
 *     caller owns every buffer, and the library keeps no pointer after a call
 *     returns.  Tensors are dense and row-major in the layouts given below.
 *   - dtype: MLA_DTYPE_BF16 (storage bf16, fp32 accumulation) or
 *     MLA_DTYPE_F32.  Every tensor of one call has the call's dtype, except
 *     positions / seqlens (int32) and the workspace (bytes).
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy
 *     default stream) and never synchronise the host, except
 *     mla_device_status().
 *   - Return value: MLA_OK (0) or a negative MLA_ERR_* code.  On error nothing
 *     was launched and mla_last_error() (thread-local) describes why.
 *   - Values that live on the device (positions, seqlens) are checked by the
 *     kernels: a bad value sets a bit in the library's device status word and
 *     the affected rows are skipped (append) or written as zeros (decode);
 *     mla_device_status() reports and clears the word.
 *   - Pointers must be 16-byte aligned (MLA_ERR_ALIGN otherwise).
 */
#ifndef MLA_H_
#define MLA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* mla_stream_t; /* same type as cudaStream_t */

enum {
    MLA_OK = 0,
    MLA_ERR_ARG = -1,         /* NULL pointer, negative size, bad enum */
    MLA_ERR_SHAPE = -2,       /* dimensions outside what an entry point supports */
    MLA_ERR_ALIGN = -3,       /* pointer or stride not 16-byte aligned */
    MLA_ERR_CUDA = -4,        /* a CUDA runtime/driver call failed */
    MLA_ERR_TIMEOUT = -5,     /* a device-side wait gave up (see mla_device_status) */
    MLA_ERR_DEVICE = -6,      /* device status word non-zero (bad positions/seqlens) */
    MLA_ERR_WORKSPACE = -7,   /* workspace NULL or smaller than mla_workspace_bytes() */
    MLA_ERR_UNSUPPORTED = -8  /* a forced path cannot run this shape / device */
};

enum { MLA_DTYPE_BF16 = 0, MLA_DTYPE_F32 = 1 };

/* Head geometry.  V3 values: H=128, d_c=512, d_r=64, d_n=128, d_v=128
 * (ailearn.mscapital.top/deepseek-v3.html, configuration table, row "MLA").
 * rope_base: RoPE frequency base (10000).  softmax_scale: 0 selects
 * 1/sqrt(d_n + d_r). */
typedef struct {
    int32_t H, d_c, d_r, d_n, d_v;
    int32_t dtype;
    float rope_base;
    float softmax_scale;
} mla_dims_t;

/* The compressed KV cache: B sequences x T_max rows; row t of sequence b
 * starts at data + b*stride_b + t*stride_t (strides in ELEMENTS) and holds
 * d_c latent values followed by d_r RoPE-key values already rotated at
 * position t.  stride_t >= d_c + d_r; strides*elem_size multiples of 16. */
typedef struct {
    void* data;
    int32_t B, T_max;
    int64_t stride_b, stride_t;
} mla_cache_t;

/* Device status bits (mla_device_status). */
enum {
    MLA_STATUS_BAD_POS = 1,     /* append: pos[b] < 0 or pos[b] + n_tok > T_max */
    MLA_STATUS_BAD_SEQLEN = 2,  /* decode: seqlens[b] < q_len or > T_max */
    MLA_STATUS_TIMEOUT = 4,     /* a bounded device-side wait expired */
    MLA_STATUS_NONFINITE = 8    /* packed append: a latent was NaN, infinite or larger than 13440 */
};

/* ---------------------------------------------------------------- a1: append
 * Write n_tok new tokens per sequence into the cache (092 page, section 二
 * "MLA：缓存压缩后的历史": the cache keeps c_KV and the RoPE key).
 *   c_kv   [B][n_tok][d_c]   latent of each new token
 *   k_rope [B][n_tok][d_r]   UN-rotated RoPE key; rotated here at its position
 *   pos    [B] int32         position of the first new token of sequence b
 * Row pos[b]+i of sequence b becomes [c_kv[b][i] || RoPE(k_rope[b][i], pos[b]+i)].
 * Rows with an out-of-range position are skipped and flag MLA_STATUS_BAD_POS. */
int mla_append_cache(const mla_dims_t* dims, const void* c_kv, const void* k_rope,
                     const int32_t* pos, int32_t B, int32_t n_tok,
                     const mla_cache_t* cache, mla_stream_t stream);

/* Bytes of scratch mla_decode / mla_attend_latent need for this shape on the
 * current device (depends on the SM count, not on the sequence lengths). */
size_t mla_workspace_bytes(const mla_dims_t* dims, int32_t B, int32_t q_len);

/* ---------------------------------------------------------------- decode
 * One absorbed-MLA decode step for B sequences with q_len query tokens each
 * (q_len = 1 plain decode; 2..16 speculative verify, causal among the new
 * tokens).  seqlens[b] counts cached tokens INCLUDING the q_len new ones,
 * which must already be appended; query i sits at position
 * m = seqlens[b] - q_len + i and attends to keys 0..m.  (The rows of later
 * new tokens get the weight 0; NaN or infinite latents there still reach the
 * earlier queries on the sm_100a path.)
 *   q_nope [B][q_len][H][d_n]   content query
 *   q_rope [B][q_len][H][d_r]   UN-rotated RoPE query (rotated here at m)
 *   W_UK   [H][d_n][d_c]        k_C = W_UK[h] c      (U in R^{d_h x d_c})
 *   W_UV   [H][d_v][d_c]        v   = W_UV[h] c
 *   out    [B][q_len][H][d_v]   written
 *   workspace: device scratch of at least mla_workspace_bytes(), 16-byte
 *   aligned; the library rounds its base up to 256 bytes inside the buffer
 *   (mla_workspace_bytes() includes that slack).  The call owns it until the
 *   stream reaches the end of the call.
 * Steps: absorb (a2), attend in latent space (a3+a4), project (a5). */
int mla_decode(const mla_dims_t* dims, const void* q_nope, const void* q_rope,
               const void* W_UK, const void* W_UV, const mla_cache_t* cache,
               const int32_t* seqlens, int32_t B, int32_t q_len, void* out,
               void* workspace, size_t workspace_bytes, mla_stream_t stream);

/* Execution options for tests, tuning and profiling.
 *   path: 0 = auto (sm_100a tensor-core kernels for bf16 V3 geometry, generic
 *         CUDA kernels otherwise), 1 = force the tensor-core path
 *         (MLA_ERR_UNSUPPORTED if it cannot run), 2 = force the generic path.
 *   num_pairs: CTA pairs (clusters) of the attention grid (0 = one per two SMs;
 *         larger values are capped to that, the clusters that fit on the
 *         device at once, for which mla_workspace_bytes() sizes the scratch).
 *   overhead_tiles: scheduling cost charged per query token (each of the
 *         B * q_len tokens is scheduled on its own), in 64-key tiles
 *         (negative = default, 2).  Refused where all sequences' tiles and
 *         charges could pass 2^24.
 *   min_tiles: smallest piece of a token's keys one cluster takes, in 64-key tiles
 *         (0 = default, 2); larger values mean fewer split partials to merge.
 *         A batch whose sequences all have the same length is cut at sequence
 *         boundaries when that costs at most a quarter more per cluster group
 *         than an even split.
 *   events / n_events: optional caller-created cudaEvent_t handles; when
 *         n_events >= MLA_NUM_EVENTS, mla_decode_ex records them on `stream`
 *         at the stage boundaries listed below, so a caller can time each
 *         kernel with cudaEventElapsedTime.  The library does not own them.
 *   wait_limit_ns: time limit of each device-side barrier wait of the
 *         attention kernel (0 = default, 2 s).  A wait that runs out sets
 *         MLA_STATUS_TIMEOUT; the kernel then stops, drains what it has in
 *         flight and exits, leaving the context usable.
 *   withhold_tile: test hook for that path; 0 = off.  A value k > 0 makes
 *         the attention kernel's loader stop before the k-th 64-key tile of
 *         each cluster, so a bounded wait runs out and the call reports
 *         MLA_STATUS_TIMEOUT (the result is then undefined).
 *   All-zero options are valid (overhead_tiles 0 charges nothing per sequence). */
typedef struct {
    int32_t path;
    int32_t num_pairs;
    int32_t overhead_tiles;
    int32_t min_tiles;
    int32_t n_events;
    void* const* events;
    int64_t wait_limit_ns;
    int32_t withhold_tile;
    int32_t reserved;
} mla_decode_opts_t;

/* Event slots recorded by mla_decode_ex (sm_100a path; the generic path
 * records 0, 1 before/after absorb and 5 at the end, with 2..4 after attend). */
enum {
    MLA_EV_START = 0,        /* before the absorb GEMM */
    MLA_EV_ABSORB_DONE = 1,  /* after absorb (before the split planner) */
    MLA_EV_ATTEND_BEGIN = 2, /* before the attention kernel */
    MLA_EV_ATTEND_END = 3,   /* after the attention kernel (before the split combine) */
    MLA_EV_COMBINE_DONE = 4, /* after the split combine (before W_UV) */
    MLA_EV_END = 5,          /* after the W_UV projection */
    MLA_NUM_EVENTS = 6
};

int mla_decode_ex(const mla_dims_t* dims, const void* q_nope, const void* q_rope,
                  const void* W_UK, const void* W_UV, const mla_cache_t* cache,
                  const int32_t* seqlens, int32_t B, int32_t q_len, void* out,
                  void* workspace, size_t workspace_bytes,
                  const mla_decode_opts_t* opts, mla_stream_t stream);

/* ---------------------------------------------------------------- no-allocation decode
 * The same decode step as mla_decode for callers that cannot allocate device
 * memory: code whose device memory is owned by another allocator (a server or
 * framework that does not let plug-ins call cudaMalloc), or a serving loop
 * that must not allocate after start-up because cudaMalloc / cudaFree can
 * synchronise the device.  The paper has no counterpart; this is an
 * interface convenience of this library.
 *
 * Arguments, layouts and results are those of mla_decode, without the
 * workspace: the scratch is a fixed 64 MiB array inside the library's device
 * image, which every GPU that loads the library keeps until the process
 * exits.  A batch whose mla_workspace_bytes() exceeds 64 MiB is rejected with
 * MLA_ERR_WORKSPACE before anything is launched; on a 148-SM B200 the limit
 * is B * q_len <= 88 query tokens (88 sequences at q_len = 1, 44 at
 * q_len = 2, 22 at q_len = 4).  The call allocates nothing
 * and calls no allocating routine.
 *
 * The first call on each device looks up the array's device address
 * (cudaGetSymbolAddress, with that device current); make that first call
 * before any stream capture.  All calls on a device share the one array and
 * it keeps the last call's contents (nothing needs to start at zero); calls
 * that overlap on the GPU, on different streams or threads, race on it and
 * must be ordered by the caller. */
int mla_decode_no_alloc(const mla_dims_t* dims, const void* q_nope, const void* q_rope,
                        const void* W_UK, const void* W_UV, const mla_cache_t* cache,
                        const int32_t* seqlens, int32_t B, int32_t q_len, void* out,
                        mla_stream_t stream);

/* ---------------------------------------------------------------- steps
 * The three stages of mla_decode, callable one by one (same layouts).
 *
 * a2: q_hat[b][i][h] = [ W_UK[h]^T q_nope[b][i][h]  ||  RoPE(q_rope[b][i][h], m) ]
 *     q_hat [B][q_len][H][d_c + d_r], dtype of the call. */
int mla_absorb_query(const mla_dims_t* dims, const void* q_nope, const void* q_rope,
                     const void* W_UK, const int32_t* seqlens, int32_t B, int32_t q_len,
                     void* q_hat, const mla_decode_opts_t* opts, mla_stream_t stream);

/* a3+a4: scores s_j = softmax_scale * (q_hat . cache_row_j) over keys
 * 0..m, softmax, o_lat = sum_j p_j c_KV,j.  o_lat [B][q_len][H][d_c]. */
int mla_attend_latent(const mla_dims_t* dims, const void* q_hat, const mla_cache_t* cache,
                      const int32_t* seqlens, int32_t B, int32_t q_len, void* o_lat,
                      void* workspace, size_t workspace_bytes,
                      const mla_decode_opts_t* opts, mla_stream_t stream);

/* a5: out[r][h] = W_UV[h] o_lat[r][h] for the `rows` = B*q_len query tokens. */
int mla_project_out(const mla_dims_t* dims, const void* o_lat, const void* W_UV,
                    int32_t rows, void* out, const mla_decode_opts_t* opts,
                    mla_stream_t stream);

/* ---------------------------------------------------------------- projections around the decode
 * Both are dense bf16 contractions on the tensor cores (split over K so that
 * a few hundred tokens still spread the weight read over every SM); both
 * need bf16, the V3 head geometry (d_c 512, d_r 64, H 128, d_v 128) and a
 * compute-capability 10.0 device (MLA_ERR_UNSUPPORTED otherwise), and
 * d_model a multiple of 64.  Each takes a workspace (fp32 split partials)
 * of the size its *_workspace_bytes() returns, 16-byte aligned, owned by
 * the call until the stream reaches its end.
 *
 * Cache append from the attention block's input (a1 with the projections
 * that produce its inputs fused in):
 *   row pos[b]+i of sequence b = [ RMSNorm_gamma(W_DKV x[b][i]) || RoPE(W_KR x[b][i], pos[b]+i) ]
 * (m.lsln.cn/news/222502 section 2.2: c^KV = W^DKV h; section 1: RMSNorm,
 *  rms_norm_eps 1e-6 in its configuration block; 092 page, section 二: the
 *  cache keeps the latent and the decoupled RoPE key;
 *  ailearn.mscapital.top MLA panel: the hidden state is projected to c_KV
 *  and k_R).  The RMSNorm is taken over the d_c latent values in fp32.
 *   x      [B][n_tok][d_model]   block input (after the block's own pre-norm)
 *   W_A    [d_c + d_r][d_model]  rows 0..d_c-1 hold W_DKV, rows d_c.. hold W_KR
 *   gamma  [d_c]                 RMSNorm gain of the latent
 *   pos    [B] int32             position of the first new token of sequence b
 * Rows with an out-of-range position are skipped and set MLA_STATUS_BAD_POS. */
size_t mla_append_from_hidden_workspace_bytes(const mla_dims_t* dims, int32_t B, int32_t n_tok, int32_t d_model);
int mla_append_from_hidden(const mla_dims_t* dims, const void* x, const void* W_A, const void* gamma,
                           const int32_t* pos, int32_t B, int32_t n_tok, int32_t d_model,
                           const mla_cache_t* cache, void* workspace, size_t workspace_bytes,
                           mla_stream_t stream);

/* Output projection of the attention block: y[r] = W_O out[r], where out[r]
 * is a decode output row viewed as H * d_v values (head-major)
 * (ailearn.mscapital.top MLA panel: aggregate in latent space, then W_UV and
 * the output projection; taojin168.com forum page, section 2.1, the MLA
 * steps' last step: an output projection maps the attention output back to
 * the model width).
 *   attn_out [rows][H * d_v]     e.g. mla_decode's out, [B * q_len][H][d_v]
 *   W_O      [d_model][H * d_v]
 *   y        [rows][d_model]     written */
size_t mla_output_projection_workspace_bytes(const mla_dims_t* dims, int32_t rows, int32_t d_model);
int mla_output_projection(const mla_dims_t* dims, const void* attn_out, const void* W_O, int32_t rows,
                          int32_t d_model, void* y, void* workspace, size_t workspace_bytes,
                          mla_stream_t stream);

/* ---------------------------------------------------------------- 4-bit cache
 * The latents of a token in 4 bits each with one 8-bit scale for every 16 of
 * them, and the rotated RoPE key unquantised: 416 bytes a token in bf16 V3
 * geometry instead of 1152, so 2.8 times the history in the same memory.
 * A packed cache is an mla_cache_t whose elements are BYTES: strides in
 * bytes, multiples of 16, stride_t >= mla_packed_row_bytes(); d_c must be a
 * multiple of 16.  A row is
 *   bytes [0, d_c/2)               codes n = q + 8, q in -7..7: in 32-bit word w, element 8w+2j
 *                                  in bits 4j..4j+3, element 8w+2j+1 in bits 16+4j..19+4j
 *   bytes [d_c/2, d_c/2 + d_c/16)  scales, byte e*8+m standing for 2^(e-21) (1 + m/8)
 *   from there, rounded up to 16   the RoPE key in the call's dtype
 * and stands for the latents q * scale, which are exact in bf16.  Rows that
 * hold no token may hold any bytes. */
size_t mla_packed_row_bytes(const mla_dims_t* dims);

/* mla_append_cache for a packed cache: the latents of a group of 16 are
 * rounded to the nearest of -7..7 times its scale (half to even), the
 * smallest scale that is not below max|x| / 7.
 *   pos   [B] int32   position of the first new token (its RoPE angle)
 *   rows  [B] int32   row it is written to; NULL: pos.  They differ once
 *                     rows have been evicted.
 * A sequence whose rows or positions are out of range is skipped and flags
 * MLA_STATUS_BAD_POS.  The key is stored as it is, NaN and infinities too,
 * without a flag.  A NaN latent is stored as 0 and one above 13440 (the
 * largest scale times 7) as 13440; both flag MLA_STATUS_NONFINITE. */
int mla_append_packed(const mla_dims_t* dims, const void* c_kv, const void* k_rope, const int32_t* pos,
                      const int32_t* rows, int32_t B, int32_t n_tok, const mla_cache_t* cache, mla_stream_t stream);

/* mla_append_cache with the row apart from the position, for a full-width
 * cache from which rows have been evicted (arguments as above). */
int mla_append_rows(const mla_dims_t* dims, const void* c_kv, const void* k_rope, const int32_t* pos,
                    const int32_t* rows, int32_t B, int32_t n_tok, const mla_cache_t* cache, mla_stream_t stream);

/* Rows rows[b] .. rows[b] + n_tok - 1 of a packed cache as full-width rows,
 * out [B][n_tok][d_c + d_r]: what a full-width cache of the same tokens
 * would hold after quantisation.  Rows out of range are written as zeros and flag
 * MLA_STATUS_BAD_POS. */
int mla_load_packed(const mla_dims_t* dims, const mla_cache_t* cache, const int32_t* rows, int32_t B, int32_t n_tok,
                    void* out, mla_stream_t stream);

/* Bytes of scratch mla_decode_packed / mla_attend_packed need. */
size_t mla_packed_workspace_bytes(const mla_dims_t* dims, int32_t B, int32_t q_len);

/* mla_attend_latent over a packed cache.  lse [B][q_len][H] fp32 (may be
 * NULL) receives the natural log of the sum over keys of exp(s_j), -infinity
 * for a sequence with an invalid length and where every score is -infinity
 * (o_lat is zero there).  A NaN among a query's scores, or +infinity, makes
 * its o_lat and its lse NaN.  Of the options, path, num_pairs,
 * overhead_tiles and min_tiles (both in 128-key tiles here, 1 by default),
 * wait_limit_ns and withhold_tile apply. */
int mla_attend_packed(const mla_dims_t* dims, const void* q_hat, const mla_cache_t* cache, const int32_t* seqlens,
                      int32_t B, int32_t q_len, void* o_lat, float* lse, void* workspace, size_t workspace_bytes,
                      const mla_decode_opts_t* opts, mla_stream_t stream);

/* mla_decode over a packed cache.  seqlens[b] counts the rows of the cache,
 * n_seen[b] the tokens the sequence has had (both including the q_len new
 * ones): query i sits at position n_seen[b] - q_len + i.  n_seen may be NULL
 * where no row has been evicted (then it is seqlens); one below q_len flags
 * MLA_STATUS_BAD_SEQLEN, and that sequence's result has no meaning.  q_hat
 * [B][q_len][H][d_c + d_r] and lse [B][q_len][H] receive the folded queries
 * and the log-sum-exps, for mla_accumulate_weights; either may be NULL. */
int mla_decode_packed(const mla_dims_t* dims, const void* q_nope, const void* q_rope, const void* W_UK,
                      const void* W_UV, const mla_cache_t* cache, const int32_t* seqlens, const int32_t* n_seen,
                      int32_t B, int32_t q_len, void* out, void* q_hat, float* lse, void* workspace,
                      size_t workspace_bytes, const mla_decode_opts_t* opts, mla_stream_t stream);

/* ---------------------------------------------------------------- eviction by accumulated attention weight
 * A cache kept within a budget of rows: after each step every row's
 * attention weight is added to a running sum, and when a sequence outgrows
 * the budget the rows with the least are dropped.  Rows keep their rotated keys, so
 * after an eviction a sequence's row count and its token count differ:
 * append with mla_append_rows / mla_append_packed, fold the queries with the
 * token counts (mla_absorb_query's seqlens, mla_decode_packed's n_seen) and
 * attend with the row counts. */
enum { MLA_CACHE_FULL = 0, MLA_CACHE_PACKED = 1 }; /* cache_format */

/* mla_attend_latent that also writes the log-sum-exps, as mla_attend_packed does (lse not NULL).  What the rows of later
 * new tokens hold does not reach a query here. */
int mla_attend_latent_lse(const mla_dims_t* dims, const void* q_hat, const mla_cache_t* cache, const int32_t* seqlens,
                          int32_t B, int32_t q_len, void* o_lat, float* lse, void* workspace, size_t workspace_bytes,
                          const mla_decode_opts_t* opts, mla_stream_t stream);

/* weights[b][t] = decay * prev[b][t] + sum_{i,h} exp(softmax_scale * q_hat[b][i][h] . row_t - lse[b][i][h])
 * for the rows t < seqlens[b] (query i counts where it sees the row; a row of lse that is -infinity counts nothing).
 *   lse     [B][q_len][H] fp32   of the same step over the same cache
 *   prev    [B][weights_stride] fp32, may be weights itself, or NULL (zero)
 *   weights [B][weights_stride] fp32; entries of rows >= seqlens[b], and of a
 *           sequence with an invalid length (flags MLA_STATUS_BAD_SEQLEN), are left as they were
 * weights_stride >= T_max.  The same call gives the same sums (no atomics); the order in which
 * several queries' parts are added depends on B, q_len, T_max, the cache's format and the device's size, not on the lengths.
 * How the work is split goes by T_max, as the lengths lie on the device: in a cache much longer than its sequences, give any
 * bound on the lengths as T_max (1 x 600 rows, 16 queries: 13 us with 600, 56 to 64 us with 131072).
 * prev and weights must not overlap otherwise.  Of the options, path,
 * wait_limit_ns and withhold_tile apply. */
int mla_accumulate_weights(const mla_dims_t* dims, const void* q_hat, const float* lse, const mla_cache_t* cache,
                           int32_t cache_format, const int32_t* seqlens, int32_t B, int32_t q_len, float decay,
                           const float* prev, float* weights, int64_t weights_stride, const mla_decode_opts_t* opts,
                           mla_stream_t stream);

/* Cuts every sequence of more than `budget` rows down to budget rows: its
 * first n_sink, its last n_recent, and of the rows between the
 * budget - n_sink - n_recent with the largest weights (equal weights: the
 * lower row; a NaN counts as less than any number).  The kept rows, in their
 * order, become rows 0.. of out_cache, their weights out_weights[b][0..], and
 * out_seqlens[b] their number; shorter sequences are kept whole.
 *   kept  [B][budget] int32, may be NULL: the kept rows' indexes, -1 past their number
 * out_cache may be the cache itself, out_weights weights, out_seqlens seqlens
 * (eviction in place); other overlaps of these pairs are refused, and so is a
 * budget above 2^30.  Rows of out_cache and entries of
 * out_weights past the kept ones are left as they were: before such a row is
 * appended to again, the caller sets its weight to zero.  A sequence with a
 * negative length or one above T_max keeps nothing and flags
 * MLA_STATUS_BAD_SEQLEN.  Here too a bound on the lengths may be given as
 * T_max (64 x 4096 rows are selected in 18 us with 4096, in 92 us with
 * 131072).  The workspace is of mla_evict_workspace_bytes() bytes, 16-byte
 * aligned, the call's until the stream reaches its end.
 * In place, the parts of a sequence wait for one another; a wait that runs
 * out flags MLA_STATUS_TIMEOUT, and the cache, its weights and lengths are
 * then undefined (parts have moved, and the lengths count the kept rows). */
size_t mla_evict_workspace_bytes(const mla_dims_t* dims, int32_t cache_format, int32_t B, int32_t budget);
int mla_evict(const mla_dims_t* dims, const mla_cache_t* cache, int32_t cache_format, const float* weights,
              int64_t weights_stride, const int32_t* seqlens, int32_t B, int32_t budget, int32_t n_sink,
              int32_t n_recent, const mla_cache_t* out_cache, float* out_weights, int64_t out_weights_stride,
              int32_t* out_seqlens, int32_t* kept, void* workspace, size_t workspace_bytes, mla_stream_t stream);

/* mla_evict with options (NULL: defaults).  wait_limit_ns applies, and withhold_tile as a test hook: a value k > 0 keeps
 * the k-th part of each sequence from being announced, so that the parts which wait for it in place run out. */
int mla_evict_ex(const mla_dims_t* dims, const mla_cache_t* cache, int32_t cache_format, const float* weights,
                 int64_t weights_stride, const int32_t* seqlens, int32_t B, int32_t budget, int32_t n_sink,
                 int32_t n_recent, const mla_cache_t* out_cache, float* out_weights, int64_t out_weights_stride,
                 int32_t* out_seqlens, int32_t* kept, void* workspace, size_t workspace_bytes,
                 const mla_decode_opts_t* opts, mla_stream_t stream);

/* ---------------------------------------------------------------- status */

/* Synchronises `stream`, returns the device status word in *status (bits
 * MLA_STATUS_*) and clears it.  Returns MLA_OK, MLA_ERR_CUDA, or
 * MLA_ERR_DEVICE when the word was non-zero. */
int mla_device_status(mla_stream_t stream, int32_t* status);

/* Description of the last error on this host thread ("" if none). */
const char* mla_last_error(void);

/* Name of the path the last mla_decode* / step call on this thread used:
 * "sm100" or "generic". */
const char* mla_last_path(void);

/* ABI version (major*100 + minor). */
int mla_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MLA_H_ */
