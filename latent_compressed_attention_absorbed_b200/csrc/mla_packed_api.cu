// C entry points of the 4-bit cache, the accumulated attention weights and
// the eviction (declared in include/mla.h): argument checks, path selection
// and workspace carving.
#include <cuda_runtime.h>
#include <math.h>

#include "mla_internal.h"
#include "mla_packed_internal.h"

namespace mla {
namespace {

int cuda_error(cudaError_t e, const char* what) {
    return e == cudaSuccess ? MLA_OK : set_error(MLA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

int check_packed_dims(const Problem& p) {
    if (p.d_c % kPackGroup)
        return set_error(MLA_ERR_SHAPE, "a packed cache needs d_c a multiple of %d, got %d", kPackGroup, p.d_c);
    return MLA_OK;
}

// The packed cache: bytes, so strides are bytes.
int check_packed_cache(const Problem& p, const mla_cache_t* c, int B, CacheView* v) {
    int rc = check_packed_dims(p);
    if (rc) return rc;
    if (!c || !c->data) return set_error(MLA_ERR_ARG, "cache or cache->data is NULL");
    if (!aligned16(c->data)) return set_error(MLA_ERR_ALIGN, "cache->data must be 16-byte aligned");
    if (c->B < B) return set_error(MLA_ERR_SHAPE, "cache holds %d sequences, call needs %d", c->B, B);
    if (c->T_max <= 0) return set_error(MLA_ERR_SHAPE, "cache T_max must be positive");
    const int64_t row = packed_layout(p.d_c, p.d_r, (int)elem_size(p)).bytes;
    if (c->stride_t < row)
        return set_error(MLA_ERR_SHAPE, "cache stride_t %lld < packed row of %lld bytes", (long long)c->stride_t, (long long)row);
    if (c->stride_b < c->stride_t * (int64_t)c->T_max && c->B > 1)
        return set_error(MLA_ERR_SHAPE, "cache stride_b smaller than T_max * stride_t");
    if (c->stride_t % 16 || c->stride_b % 16)
        return set_error(MLA_ERR_ALIGN, "cache strides must be multiples of 16 bytes");
    v->data = c->data;
    v->T_max = c->T_max;
    v->stride_b = c->stride_b;
    v->stride_t = c->stride_t;
    return MLA_OK;
}

int check_any_cache(const Problem& p, const mla_cache_t* c, int format, int B, CacheView* v) {
    if (format == MLA_CACHE_PACKED) return check_packed_cache(p, c, B, v);
    if (format == MLA_CACHE_FULL) return check_cache(p, c, B, v);
    return set_error(MLA_ERR_ARG, "cache format must be MLA_CACHE_FULL or MLA_CACHE_PACKED, got %d", format);
}

int check_query(const mla_dims_t* dims, int32_t B, int32_t q_len, Problem* p) {
    set_error(MLA_OK, "%s", "");
    int rc = check_dims(dims, p);
    if (rc) return rc;
    if (B < 0 || q_len < 1 || q_len > 16) return set_error(MLA_ERR_ARG, "need B >= 0 and 1 <= q_len <= 16");
    p->B = B;
    p->q_len = q_len;
    return MLA_OK;
}

int write_rows(const mla_dims_t* dims, bool packed, const void* c_kv, const void* k_rope, const int32_t* pos,
               const int32_t* rows, int32_t B, int32_t n_tok, const mla_cache_t* cache, mla_stream_t stream) {
    set_error(MLA_OK, "%s", "");
    Problem p;
    int rc = check_dims(dims, &p);
    if (rc) return rc;
    if (packed && (rc = check_packed_dims(p))) return rc;
    if (B < 0 || n_tok < 0) return set_error(MLA_ERR_ARG, "B and n_tok must be >= 0");
    if (B == 0 || n_tok == 0) return MLA_OK;
    if (!c_kv || (!k_rope && p.d_r > 0) || !pos) return set_error(MLA_ERR_ARG, "NULL tensor pointer");
    if (!aligned16(c_kv) || !aligned16(k_rope) || !aligned4(pos) || !aligned4(rows))
        return set_error(MLA_ERR_ALIGN, "misaligned pointer");
    CacheView cv;
    rc = check_any_cache(p, cache, packed ? MLA_CACHE_PACKED : MLA_CACHE_FULL, B, &cv);
    if (rc) return rc;
    p.B = B;
    int* status = device_status_ptr();
    if (!status) return set_error(MLA_ERR_CUDA, "no CUDA device / status word");
    return cuda_error(rows_append(p, packed, c_kv, k_rope, pos, rows, n_tok, cv, status, (cudaStream_t)stream),
                      "append launch");
}

struct PackedDecodeLayout {
    size_t q_hat, o_lat, attend, total;
};

// The tensor-core attention's part is always counted where it can run, so that
// one size serves every option.
PackedDecodeLayout packed_decode_layout(const Problem& p) {
    Carve c(nullptr);
    PackedDecodeLayout L;
    const size_t U = (size_t)p.B * p.q_len * p.H;
    L.q_hat = c.off;
    c.take(U * (p.d_c + p.d_r) * elem_size(p));
    L.o_lat = c.off;
    c.take(U * p.d_c * elem_size(p));
    L.attend = c.off;
    if (sm100_supported(p, p.q_len)) c.take(sm100_attend_workspace_bytes(p, sm100_default_pairs()) + kWsAlign);
    L.total = c.off;
    return L;
}

// mla_attend_packed; n_seen (NULL: not checked) as mla_decode_packed has it.
int attend_packed(const mla_dims_t* dims, const void* q_hat, const mla_cache_t* cache, const int32_t* seqlens,
                  const int32_t* n_seen, int32_t B, int32_t q_len, void* o_lat, float* lse, void* workspace,
                  size_t workspace_bytes, const mla_decode_opts_t* opts, mla_stream_t stream) {
    Problem p;
    int rc = check_query(dims, B, q_len, &p);
    if (rc) return rc;
    if ((rc = check_packed_dims(p))) return rc;
    if (B == 0) return MLA_OK;
    if (!q_hat || !seqlens || !o_lat) return set_error(MLA_ERR_ARG, "NULL tensor pointer");
    if (!aligned16(q_hat) || !aligned16(o_lat) || !aligned4(seqlens) || !aligned4(lse))
        return set_error(MLA_ERR_ALIGN, "misaligned pointer");
    CacheView cv;
    rc = check_packed_cache(p, cache, B, &cv);
    if (rc) return rc;
    bool fast;
    rc = choose_path(p, q_len, opts, &fast);
    if (rc || (rc = check_split(p, cv.T_max, opts))) return rc;
    int* status = device_status_ptr();
    if (!status) return set_error(MLA_ERR_CUDA, "no CUDA device / status word");
    if (!fast)
        return cuda_error(generic_attend_rows(p, true, q_hat, cv, seqlens, n_seen, o_lat, lse, status, (cudaStream_t)stream),
                          "packed attend launch");
    const int pairs = pairs_for(opts);
    const size_t need = sm100_attend_workspace_bytes(p, pairs) + kWsAlign;
    if (!workspace || workspace_bytes < need || !aligned16(workspace))
        return set_error(MLA_ERR_WORKSPACE, "packed attend workspace needs %zu bytes (16-byte aligned), got %zu", need,
                         workspace_bytes);
    workspace = align_ws(workspace, &workspace_bytes);
    return cuda_error(sm100_attend_packed(p, q_hat, cv, seqlens, n_seen, o_lat, lse, workspace, workspace_bytes, pairs, status,
                                          opts, (cudaStream_t)stream),
                      "packed attend launch");
}

// The bytes a view can touch: B sequences of `rows` rows of `row` bytes.
struct Span {
    uintptr_t at;
    int64_t B, stride_b, rows, stride_t, row;
    int64_t each() const { return (rows - 1) * stride_t + row; }  // bytes from a sequence's start to its end
    uintptr_t end() const { return at + (uintptr_t)((B - 1) * stride_b + each()); }
    // Whether two views may share a byte.  Views of one array that lie between each
    // other do not: in a common period the bytes of one lie behind those of the other.
    bool overlaps(const Span& o) const {
        if (end() <= o.at || o.end() <= at) return false;
        auto apart = [](int64_t d, int64_t period, int64_t n, int64_t n_other) {
            d = (d % period + period) % period;  // where the other's bytes start in this one's period
            return d >= n && d + n_other <= period;
        };
        const int64_t d = (int64_t)(o.at - at);
        if (B > 1 && o.B > 1 && stride_b == o.stride_b && apart(d, stride_b, each(), o.each())) return false;
        const bool rows_in_step = stride_t == o.stride_t && (B == 1 || stride_b % stride_t == 0) &&
                                  (o.B == 1 || o.stride_b % stride_t == 0);
        return !(rows_in_step && apart(d, stride_t, row, o.row));
    }
};
Span span_of(const void* p, int64_t B, int64_t stride_b, int64_t rows, int64_t stride_t, int64_t row) {
    return {reinterpret_cast<uintptr_t>(p), B, stride_b, rows, stride_t, row};
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

size_t mla_packed_row_bytes(const mla_dims_t* dims) {
    Problem p;
    if (check_dims(dims, &p) || check_packed_dims(p)) return 0;
    return (size_t)packed_layout(p.d_c, p.d_r, (int)elem_size(p)).bytes;
}

int mla_append_packed(const mla_dims_t* dims, const void* c_kv, const void* k_rope, const int32_t* pos,
                      const int32_t* rows, int32_t B, int32_t n_tok, const mla_cache_t* cache, mla_stream_t stream) {
    return write_rows(dims, true, c_kv, k_rope, pos, rows, B, n_tok, cache, stream);
}

int mla_append_rows(const mla_dims_t* dims, const void* c_kv, const void* k_rope, const int32_t* pos,
                    const int32_t* rows, int32_t B, int32_t n_tok, const mla_cache_t* cache, mla_stream_t stream) {
    return write_rows(dims, false, c_kv, k_rope, pos, rows, B, n_tok, cache, stream);
}

int mla_load_packed(const mla_dims_t* dims, const mla_cache_t* cache, const int32_t* rows, int32_t B, int32_t n_tok,
                    void* out, mla_stream_t stream) {
    set_error(MLA_OK, "%s", "");
    Problem p;
    int rc = check_dims(dims, &p);
    if (rc) return rc;
    if ((rc = check_packed_dims(p))) return rc;
    if (B < 0 || n_tok < 0) return set_error(MLA_ERR_ARG, "B and n_tok must be >= 0");
    if (B == 0 || n_tok == 0) return MLA_OK;
    if (!rows || !out) return set_error(MLA_ERR_ARG, "NULL tensor pointer");
    if (!aligned16(out) || !aligned4(rows)) return set_error(MLA_ERR_ALIGN, "misaligned pointer");
    CacheView cv;
    rc = check_packed_cache(p, cache, B, &cv);
    if (rc) return rc;
    p.B = B;
    int* status = device_status_ptr();
    if (!status) return set_error(MLA_ERR_CUDA, "no CUDA device / status word");
    return cuda_error(packed_load(p, cv, rows, n_tok, out, status, (cudaStream_t)stream), "load launch");
}

size_t mla_packed_workspace_bytes(const mla_dims_t* dims, int32_t B, int32_t q_len) {
    Problem p;
    if (check_query(dims, B, q_len, &p) || check_packed_dims(p)) return 0;
    return packed_decode_layout(p).total + kWsAlign;
}

int mla_attend_packed(const mla_dims_t* dims, const void* q_hat, const mla_cache_t* cache, const int32_t* seqlens,
                      int32_t B, int32_t q_len, void* o_lat, float* lse, void* workspace, size_t workspace_bytes,
                      const mla_decode_opts_t* opts, mla_stream_t stream) {
    return attend_packed(dims, q_hat, cache, seqlens, nullptr, B, q_len, o_lat, lse, workspace, workspace_bytes, opts, stream);
}

int mla_decode_packed(const mla_dims_t* dims, const void* q_nope, const void* q_rope, const void* W_UK,
                      const void* W_UV, const mla_cache_t* cache, const int32_t* seqlens, const int32_t* n_seen,
                      int32_t B, int32_t q_len, void* out, void* q_hat, float* lse, void* workspace,
                      size_t workspace_bytes, const mla_decode_opts_t* opts, mla_stream_t stream) {
    Problem p;
    int rc = check_query(dims, B, q_len, &p);
    if (rc) return rc;
    if ((rc = check_packed_dims(p))) return rc;
    if (B == 0) return MLA_OK;
    if (!q_nope || !q_rope || !W_UK || !W_UV || !seqlens || !out) return set_error(MLA_ERR_ARG, "NULL tensor pointer");
    if (!aligned16(q_nope) || !aligned16(q_rope) || !aligned16(W_UK) || !aligned16(W_UV) || !aligned16(out) ||
        !aligned16(q_hat) || !aligned4(seqlens) || !aligned4(n_seen) || !aligned4(lse))
        return set_error(MLA_ERR_ALIGN, "misaligned pointer");
    CacheView cv;
    rc = check_packed_cache(p, cache, B, &cv);
    if (rc || (rc = check_split(p, cv.T_max, opts))) return rc;
    const size_t need = mla_packed_workspace_bytes(dims, B, q_len);
    if (!workspace || workspace_bytes < need || !aligned16(workspace))
        return set_error(MLA_ERR_WORKSPACE, "packed decode workspace needs %zu bytes (16-byte aligned), got %zu", need,
                         workspace_bytes);
    workspace = align_ws(workspace, &workspace_bytes);
    const PackedDecodeLayout L = packed_decode_layout(p);
    char* ws = static_cast<char*>(workspace);
    void* qh = q_hat ? q_hat : ws + L.q_hat;
    void* o_lat = ws + L.o_lat;
    rc = mla_absorb_query(dims, q_nope, q_rope, W_UK, n_seen ? n_seen : seqlens, B, q_len, qh, opts, stream);
    if (rc) return rc;
    rc = attend_packed(dims, qh, cache, seqlens, n_seen, B, q_len, o_lat, lse, ws + L.attend, L.total - L.attend, opts,
                       stream);
    if (rc) return rc;
    return mla_project_out(dims, o_lat, W_UV, B * q_len, out, opts, stream);
}

int mla_attend_latent_lse(const mla_dims_t* dims, const void* q_hat, const mla_cache_t* cache, const int32_t* seqlens,
                          int32_t B, int32_t q_len, void* o_lat, float* lse, void* workspace, size_t workspace_bytes,
                          const mla_decode_opts_t* opts, mla_stream_t stream) {
    Problem p;
    int rc = check_query(dims, B, q_len, &p);
    if (rc) return rc;
    if (B == 0) return MLA_OK;
    if (!q_hat || !seqlens || !o_lat || !lse) return set_error(MLA_ERR_ARG, "NULL tensor pointer");
    if (!aligned16(q_hat) || !aligned16(o_lat) || !aligned4(seqlens) || !aligned4(lse))
        return set_error(MLA_ERR_ALIGN, "misaligned pointer");
    CacheView cv;
    rc = check_cache(p, cache, B, &cv);
    if (rc) return rc;
    bool fast;
    rc = choose_path(p, q_len, opts, &fast);
    if (rc || (rc = check_split(p, cv.T_max, opts))) return rc;
    int* status = device_status_ptr();
    if (!status) return set_error(MLA_ERR_CUDA, "no CUDA device / status word");
    if (!fast)
        return cuda_error(generic_attend_rows(p, false, q_hat, cv, seqlens, nullptr, o_lat, lse, status, (cudaStream_t)stream),
                          "attend launch");
    const int pairs = pairs_for(opts);
    const size_t need = sm100_attend_workspace_bytes(p, pairs) + kWsAlign;
    if (!workspace || workspace_bytes < need || !aligned16(workspace))
        return set_error(MLA_ERR_WORKSPACE, "attend workspace needs %zu bytes (16-byte aligned), got %zu", need,
                         workspace_bytes);
    workspace = align_ws(workspace, &workspace_bytes);
    return cuda_error(sm100_attend(p, q_hat, cv, seqlens, o_lat, workspace, workspace_bytes, pairs,
                                   opts ? opts->overhead_tiles : -1, opts ? opts->min_tiles : 0, status,
                                   (cudaStream_t)stream, nullptr, false, true, nullptr, 0, opts, lse),
                      "attend launch");
}

int mla_accumulate_weights(const mla_dims_t* dims, const void* q_hat, const float* lse, const mla_cache_t* cache,
                           int32_t cache_format, const int32_t* seqlens, int32_t B, int32_t q_len, float decay,
                           const float* prev, float* weights, int64_t weights_stride, const mla_decode_opts_t* opts,
                           mla_stream_t stream) {
    Problem p;
    int rc = check_query(dims, B, q_len, &p);
    if (rc) return rc;
    if (!(fabsf(decay) <= 3.4e38f)) return set_error(MLA_ERR_ARG, "decay must be a finite number");
    if (B == 0) return MLA_OK;
    if (!q_hat || !lse || !seqlens || !weights) return set_error(MLA_ERR_ARG, "NULL tensor pointer");
    if (!aligned16(q_hat) || !aligned4(lse) || !aligned4(seqlens) || !aligned4(prev) || !aligned4(weights))
        return set_error(MLA_ERR_ALIGN, "misaligned pointer");
    CacheView cv;
    rc = check_any_cache(p, cache, cache_format, B, &cv);
    if (rc) return rc;
    if (weights_stride < cv.T_max)
        return set_error(MLA_ERR_SHAPE, "weights_stride %lld < cache T_max %d", (long long)weights_stride, cv.T_max);
    if (prev && prev != weights &&
        span_of(prev, B, 4 * weights_stride, cv.T_max, 4, 4).overlaps(span_of(weights, B, 4 * weights_stride, cv.T_max, 4, 4)))
        return set_error(MLA_ERR_ARG, "prev overlaps weights: pass the same array, or one apart from it");
    bool fast;
    rc = choose_path(p, q_len, opts, &fast);
    if (rc) return rc;
    int* status = device_status_ptr();
    if (!status) return set_error(MLA_ERR_CUDA, "no CUDA device / status word");
    if (fast)
        return cuda_error(sm100_weights(p, cache_format == MLA_CACHE_PACKED, q_hat, lse, cv, seqlens, decay, prev, weights,
                                        weights_stride, status, opts, (cudaStream_t)stream),
                          "weights launch");
    return cuda_error(generic_weights(p, cache_format == MLA_CACHE_PACKED, q_hat, lse, cv, seqlens, decay, prev, weights,
                                      weights_stride, status, (cudaStream_t)stream),
                      "weights launch");
}

static int evict_row_bytes(const Problem& p, int format) {
    return format == MLA_CACHE_PACKED ? packed_layout(p.d_c, p.d_r, (int)elem_size(p)).bytes
                                      : (p.d_c + p.d_r) * (int)elem_size(p);
}

// Rows and chunks of rows are counted in 32 bits, with room to run past the budget by a block's threads.
static constexpr int32_t kMaxBudget = 1 << 30;

size_t mla_evict_workspace_bytes(const mla_dims_t* dims, int32_t cache_format, int32_t B, int32_t budget) {
    Problem p;
    if (check_dims(dims, &p) || B < 0 || budget < 1 || budget > kMaxBudget) return 0;
    if (cache_format != MLA_CACHE_FULL && cache_format != MLA_CACHE_PACKED) return 0;
    if (cache_format == MLA_CACHE_PACKED && check_packed_dims(p)) return 0;
    return evict_workspace(B, budget, evict_row_bytes(p, cache_format)) + kWsAlign;
}

int mla_evict(const mla_dims_t* dims, const mla_cache_t* cache, int32_t cache_format, const float* weights,
              int64_t weights_stride, const int32_t* seqlens, int32_t B, int32_t budget, int32_t n_sink,
              int32_t n_recent, const mla_cache_t* out_cache, float* out_weights, int64_t out_weights_stride,
              int32_t* out_seqlens, int32_t* kept, void* workspace, size_t workspace_bytes, mla_stream_t stream) {
    return mla_evict_ex(dims, cache, cache_format, weights, weights_stride, seqlens, B, budget, n_sink, n_recent, out_cache,
                        out_weights, out_weights_stride, out_seqlens, kept, workspace, workspace_bytes, nullptr, stream);
}

int mla_evict_ex(const mla_dims_t* dims, const mla_cache_t* cache, int32_t cache_format, const float* weights,
                 int64_t weights_stride, const int32_t* seqlens, int32_t B, int32_t budget, int32_t n_sink,
                 int32_t n_recent, const mla_cache_t* out_cache, float* out_weights, int64_t out_weights_stride,
                 int32_t* out_seqlens, int32_t* kept, void* workspace, size_t workspace_bytes,
                 const mla_decode_opts_t* opts, mla_stream_t stream) {
    set_error(MLA_OK, "%s", "");
    Problem p;
    int rc = check_dims(dims, &p);
    if (rc) return rc;
    if (B < 0 || budget < 1 || budget > kMaxBudget)
        return set_error(MLA_ERR_ARG, "need B >= 0 and 1 <= budget <= %d", kMaxBudget);
    if (n_sink < 0 || n_recent < 0 || (int64_t)n_sink + n_recent > budget)
        return set_error(MLA_ERR_ARG, "need n_sink >= 0, n_recent >= 0 and n_sink + n_recent <= budget (%d + %d, %d)", n_sink,
                         n_recent, budget);
    if (B == 0) return MLA_OK;
    if (!weights || !seqlens || !out_weights || !out_seqlens) return set_error(MLA_ERR_ARG, "NULL tensor pointer");
    if (!aligned4(weights) || !aligned4(seqlens) || !aligned4(out_weights) || !aligned4(out_seqlens) || !aligned4(kept))
        return set_error(MLA_ERR_ALIGN, "misaligned pointer");
    CacheView from, to;
    rc = check_any_cache(p, cache, cache_format, B, &from);
    if (rc) return rc;
    rc = check_any_cache(p, out_cache, cache_format, B, &to);
    if (rc) return rc;
    const int32_t most = budget < from.T_max ? budget : from.T_max;  // rows a sequence can keep
    if (to.T_max < most) return set_error(MLA_ERR_SHAPE, "out_cache T_max %d cannot hold %d kept rows", to.T_max, most);
    if (weights_stride < from.T_max || out_weights_stride < most)
        return set_error(MLA_ERR_SHAPE, "weights stride smaller than the rows it covers");
    EvictArgs a;
    a.B = B;
    a.T_max = from.T_max;
    a.budget = budget;
    a.n_sink = n_sink;
    a.n_recent = n_recent;
    a.row_bytes = evict_row_bytes(p, cache_format);
    const int64_t unit = cache_format == MLA_CACHE_PACKED ? 1 : (int64_t)elem_size(p);
    a.src = static_cast<const uint8_t*>(from.data);
    a.dst = static_cast<uint8_t*>(to.data);
    a.src_b = from.stride_b * unit;
    a.src_t = from.stride_t * unit;
    a.dst_b = to.stride_b * unit;
    a.dst_t = to.stride_t * unit;
    a.weights = weights;
    a.weights_out = out_weights;
    a.stride_w = weights_stride;
    a.stride_w_out = out_weights_stride;
    a.seqlens = seqlens;
    a.seqlens_out = out_seqlens;
    a.kept_out = kept;
    // Moving within a buffer is ordered row by row, which needs the same rows
    // under the same addresses; any other overlap would overwrite what is still to be read.
    const bool rows_same = a.src == a.dst, weights_same = a.weights == a.weights_out;
    if (rows_same ? (a.src_b != a.dst_b || a.src_t != a.dst_t)
                  : span_of(a.src, B, a.src_b, from.T_max, a.src_t, a.row_bytes)
                        .overlaps(span_of(a.dst, B, a.dst_b, to.T_max, a.dst_t, a.row_bytes)))
        return set_error(MLA_ERR_ARG, "out_cache overlaps the cache: pass the same view, or one apart from it");
    if (weights_same ? weights_stride != out_weights_stride
                     : span_of(weights, B, 4 * weights_stride, from.T_max, 4, 4)
                           .overlaps(span_of(out_weights, B, 4 * out_weights_stride, most, 4, 4)))
        return set_error(MLA_ERR_ARG, "out_weights overlaps weights: pass the same array, or one apart from it");
    if (seqlens != out_seqlens && span_of(seqlens, 1, 0, B, 4, 4).overlaps(span_of(out_seqlens, 1, 0, B, 4, 4)))
        return set_error(MLA_ERR_ARG, "out_seqlens overlaps seqlens: pass the same array, or one apart from it");
    a.in_place = rows_same || weights_same;
    a.wait_limit_ns = opts && opts->wait_limit_ns > 0 ? (uint64_t)opts->wait_limit_ns : 0;
    a.withhold_chunk = opts && opts->withhold_tile > 0 ? opts->withhold_tile - 1 : -1;
    const size_t need = evict_workspace(B, budget, a.row_bytes) + kWsAlign;
    if (!workspace || workspace_bytes < need || !aligned16(workspace))
        return set_error(MLA_ERR_WORKSPACE, "evict workspace needs %zu bytes (16-byte aligned), got %zu", need, workspace_bytes);
    workspace = align_ws(workspace, &workspace_bytes);
    a.status = device_status_ptr();
    if (!a.status) return set_error(MLA_ERR_CUDA, "no CUDA device / status word");
    return cuda_error(evict_launch(a, workspace, (cudaStream_t)stream), "evict launch");
}

}  // extern "C"
