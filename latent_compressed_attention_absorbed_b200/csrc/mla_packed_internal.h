// Internal declarations of the 4-bit cache, the accumulated attention weights
// and the eviction (not part of the C ABI).
#pragma once

#include "mla_internal.h"
#include "mla_packed.cuh"

namespace mla {

// Rows written at rows[b] + i (NULL: pos[b] + i), the key rotated at pos[b] + i.
// For a packed cache the view's strides are bytes.
cudaError_t rows_append(const Problem& p, bool packed, const void* c_kv, const void* k_rope, const int32_t* pos,
                        const int32_t* rows, int n_tok, const CacheView& cache, int* status, cudaStream_t st);
cudaError_t packed_load(const Problem& p, const CacheView& cache, const int32_t* rows, int n_tok, void* out, int* status,
                        cudaStream_t st);
// CUDA-core forms, any geometry; lse may be NULL.  n_seen (NULL: not checked):
// token counts of the queries' positions, flagged where they are too small.
cudaError_t generic_attend_rows(const Problem& p, bool packed, const void* q_hat, const CacheView& cache,
                                const int32_t* seqlens, const int32_t* n_seen, void* o_lat, float* lse, int* status,
                                cudaStream_t st);
cudaError_t generic_weights(const Problem& p, bool packed, const void* q_hat, const float* lse, const CacheView& cache,
                            const int32_t* seqlens, float decay, const float* prev, float* weights, int64_t stride_w,
                            int* status, cudaStream_t st);

// Tensor-core form (sm100_supported); the workspace is sm100_attend_workspace_bytes().
cudaError_t sm100_attend_packed(const Problem& p, const void* q_hat, const CacheView& cache, const int32_t* seqlens,
                                const int32_t* n_seen, void* o_lat, float* lse, void* workspace, size_t ws_bytes, int num_pairs, int* status,
                                const mla_decode_opts_t* opts, cudaStream_t st);

cudaError_t sm100_weights(const Problem& p, bool packed, const void* q_hat, const float* lse, const CacheView& cache,
                          const int32_t* seqlens, float decay, const float* prev, float* weights, int64_t stride_w,
                          int* status, const mla_decode_opts_t* opts, cudaStream_t st);

// Eviction: which rows stay, and the compaction.
struct EvictArgs {
    int B, T_max, budget, n_sink, n_recent;
    int row_bytes;
    const uint8_t* src;  // rows, strides in bytes
    uint8_t* dst;
    int64_t src_b, src_t, dst_b, dst_t;
    const float* weights;
    float* weights_out;
    int64_t stride_w, stride_w_out;
    const int32_t* seqlens;
    int32_t* seqlens_out;
    int32_t* kept_out;  // [B][budget], or NULL
    bool in_place;      // rows or weights are moved within their own buffer
    uint64_t wait_limit_ns;  // 0: the default
    int withhold_chunk;  // test hook (>= 0): this chunk of a sequence does not say that it is loaded (see mla.h)
    int* status;
};
size_t evict_workspace(int B, int budget, int row_bytes);
cudaError_t evict_launch(const EvictArgs& a, void* workspace, cudaStream_t st);

}  // namespace mla
