// Rows of the compressed cache, one warp each: tokens quantised into 4-bit
// rows, packed rows read back, and full-width rows written at a row index of
// their own; and the CUDA-core forms of the attention over packed rows and of
// the accumulated attention weights (any head geometry, fp32 or bf16), which
// serve the shapes the tensor-core kernels do not cover and check them.
#include <cuda_bf16.h>
#include <limits.h>
#include <math.h>

#include "mla_internal.h"
#include "mla_packed.cuh"
#include "mla_packed_internal.h"
#include "mla_rope.cuh"
#include "sm100_unpack.cuh"

namespace mla {
namespace {

__device__ __forceinline__ float ld(const float* p, size_t i) { return p[i]; }
__device__ __forceinline__ float ld(const __nv_bfloat16* p, size_t i) { return __bfloat162float(p[i]); }
__device__ __forceinline__ void st(float* p, size_t i, float v) { p[i] = v; }
__device__ __forceinline__ void st(__nv_bfloat16* p, size_t i, float v) { p[i] = __float2bfloat16_rn(v); }

// 16 consecutive elements, 16-byte aligned.
__device__ __forceinline__ void ld16(const float* p, float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(p) + i);
        x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
    }
}
__device__ __forceinline__ void ld16(const __nv_bfloat16* p, float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
            x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    }
}
__device__ __forceinline__ void st16(float* p, const float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        reinterpret_cast<float4*>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
}
__device__ __forceinline__ void st16(__nv_bfloat16* p, const float (&x)[16]) {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&v);
    }
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

constexpr int kRowWarps = 4;  // warps (rows) of a block

// The row index and position of token i of sequence b; false (and the status
// bit, once per sequence) if the new tokens do not fit.
__device__ __forceinline__ bool row_and_pos(const int32_t* pos, const int32_t* rows, int b, int i, int n_tok, int T_max,
                                            int lane, int* status, int* row, int* p) {
    const int p0 = pos[b], r0 = rows ? rows[b] : p0;
    if (p0 < 0 || p0 > INT_MAX - n_tok || r0 < 0 || r0 > T_max - n_tok) {
        if (lane == 0 && i == 0) atomicOr(status, MLA_STATUS_BAD_POS);
        return false;
    }
    *row = r0 + i;
    *p = p0 + i;
    return true;
}

// Codes and scale of the 16 latents at src.  4 bits cannot hold a NaN or an
// infinity: a NaN is stored as 0, what is above 13440 as the largest level, and
// `odd` is set.
__device__ __forceinline__ void quantise_group(const float* src, uint32_t (&w)[2], uint32_t& code, bool& odd) {
    float x[16], amax = 0.f;
    ld16(src, x);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        if (!(fabsf(x[e]) <= 13440.0f)) {
            odd = true;
            x[e] = x[e] > 0.f ? 13440.0f : (x[e] < 0.f ? -13440.0f : 0.f);
        }
        amax = fmaxf(amax, fabsf(x[e]));
    }
    code = packed_scale_code(amax);
    const float s = packed_scale(code), inv = 1.0f / s;
    w[0] = w[1] = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) w[e / 8] |= (uint32_t)(packed_quantise(x[e], s, inv) + 8) << packed_shift(e & 7);
}
__device__ __forceinline__ void quantise_group(const __nv_bfloat16* src, uint32_t (&w)[2], uint32_t& code, bool& odd) {
    uint32_t v[8];
    const uint4 lo = __ldg(reinterpret_cast<const uint4*>(src)), hi = __ldg(reinterpret_cast<const uint4*>(src) + 1);
    v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
    v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
    // magnitudes compare as integers, and a NaN is larger than an infinity
    uint32_t top = v[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int j = 1; j < 8; ++j) top = __vmaxu2(top, v[j] & 0x7FFF7FFFu);
    const uint32_t mag = max(top & 0xFFFFu, top >> 16);
    float amax = __uint_as_float(mag << 16);
    if (mag > 0x4652u) {  // 13440
        odd = true;
        amax = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t fixed = 0;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t b = (v[j] >> (16 * half)) & 0xFFFFu;
                if ((b & 0x7FFFu) > 0x7F80u) b = 0;
                else if ((b & 0x7FFFu) > 0x4652u) b = (b & 0x8000u) | 0x4652u;
                amax = fmaxf(amax, __uint_as_float((b & 0x7FFFu) << 16));
                fixed |= b << (16 * half);
            }
            v[j] = fixed;
        }
    }
    code = packed_scale_code(amax);
    const float inv = 1.0f / packed_scale(code);
    w[0] = w[1] = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {  // elements 2j and 2j + 1
        w[j / 4] |= packed_code_bf16(__uint_as_float(v[j] << 16), inv) << (4 * (j & 3));
        w[j / 4] |= packed_code_bf16(__uint_as_float(v[j] & 0xFFFF0000u), inv) << (4 * (j & 3) + 16);
    }
}

// A warp quantises one token.  Each lane owns whole groups of 16 latents (one
// each at d_c = 512), so the group's maximum needs no exchange between lanes,
// and the warp's stores of codes, scales and key are contiguous.  1152 bytes
// are read and 416 written a token in bf16; the arithmetic (five instructions
// a latent in bf16, and the rotation of the key) is kept small enough for that
// to be the bound.
template <typename T>
__global__ void __launch_bounds__(kRowWarps * 32)
    append_packed_kernel(const T* __restrict__ c_kv, const T* __restrict__ k_rope, const int32_t* __restrict__ pos,
                         const int32_t* __restrict__ rows, int64_t tokens, int n_tok, int d_c, int d_r, CacheView cache,
                         RopeTable rope, int* status) {
    const int64_t gw = (int64_t)blockIdx.x * kRowWarps + threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    if (gw >= tokens) return;
    const int b = (int)(gw / n_tok), i = (int)(gw % n_tok);
    int r, p;
    if (!row_and_pos(pos, rows, b, i, n_tok, cache.T_max, lane, status, &r, &p)) return;
    const PackedLayout l = packed_layout(d_c, d_r, sizeof(T));
    uint8_t* row = static_cast<uint8_t*>(cache.data) + (int64_t)b * cache.stride_b + (int64_t)r * cache.stride_t;
    bool odd = false;
    for (int g = lane; g < d_c / kPackGroup; g += 32) {
        uint32_t w[2], code;
        quantise_group(c_kv + gw * d_c + g * kPackGroup, w, code, odd);
        reinterpret_cast<uint2*>(row)[g] = make_uint2(w[0], w[1]);
        row[l.off_scale + g] = (uint8_t)code;
    }
    if (odd) atomicOr(status, MLA_STATUS_NONFINITE);
    const T* k = k_rope + gw * d_r;
    T* dst = reinterpret_cast<T*>(row + l.off_rope);
    for (int kk = lane; kk < d_r / 2; kk += 32) {
        float y0, y1;
        mla_rope_rotate(ld(k, 2 * kk), ld(k, 2 * kk + 1), rope.inv_freq[kk], p, &y0, &y1);
        st(dst, 2 * kk, y0);
        st(dst, 2 * kk + 1, y1);
    }
}

// Full-width rows at a row index apart from the position (a warp a token).
template <typename T>
__global__ void __launch_bounds__(kRowWarps * 32)
    append_rows_kernel(const T* __restrict__ c_kv, const T* __restrict__ k_rope, const int32_t* __restrict__ pos,
                       const int32_t* __restrict__ rows, int64_t tokens, int n_tok, int d_c, int d_r, CacheView cache,
                       RopeTable rope, int* status) {
    const int64_t gw = (int64_t)blockIdx.x * kRowWarps + threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    if (gw >= tokens) return;
    const int b = (int)(gw / n_tok), i = (int)(gw % n_tok);
    int r, p;
    if (!row_and_pos(pos, rows, b, i, n_tok, cache.T_max, lane, status, &r, &p)) return;
    T* row = static_cast<T*>(cache.data) + (int64_t)b * cache.stride_b + (int64_t)r * cache.stride_t;
    const T* src = c_kv + gw * d_c;
    if ((d_c * sizeof(T)) % 16 == 0) {
        const int n = d_c * (int)sizeof(T) / 16;
        for (int e = lane; e < n; e += 32) reinterpret_cast<uint4*>(row)[e] = __ldg(reinterpret_cast<const uint4*>(src) + e);
    } else {
        for (int e = lane; e < d_c; e += 32) row[e] = src[e];
    }
    const T* k = k_rope + gw * d_r;
    for (int kk = lane; kk < d_r / 2; kk += 32) {
        float y0, y1;
        mla_rope_rotate(ld(k, 2 * kk), ld(k, 2 * kk + 1), rope.inv_freq[kk], p, &y0, &y1);
        st(row, d_c + 2 * kk, y0);
        st(row, d_c + 2 * kk + 1, y1);
    }
}

// Packed rows as full-width rows (a warp a row): the values are exact in T.
template <typename T>
__global__ void __launch_bounds__(kRowWarps * 32)
    load_packed_kernel(CacheView cache, const int32_t* __restrict__ rows, int64_t tokens, int n_tok, int d_c, int d_r,
                       T* __restrict__ out, int* status) {
    const int64_t gw = (int64_t)blockIdx.x * kRowWarps + threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    if (gw >= tokens) return;
    const int b = (int)(gw / n_tok), i = (int)(gw % n_tok);
    T* dst = out + gw * (d_c + d_r);
    const int r0 = rows[b];
    if (r0 < 0 || r0 > cache.T_max - n_tok) {
        if (lane == 0 && i == 0) atomicOr(status, MLA_STATUS_BAD_POS);
        for (int e = lane; e < d_c + d_r; e += 32) st(dst, e, 0.f);
        return;
    }
    const PackedLayout l = packed_layout(d_c, d_r, sizeof(T));
    const uint8_t* row = static_cast<const uint8_t*>(cache.data) + (int64_t)b * cache.stride_b + (int64_t)(r0 + i) * cache.stride_t;
    const bool wide = ((d_c + d_r) * sizeof(T)) % 16 == 0;
    for (int g = lane; g < d_c / kPackGroup; g += 32) {
        const uint2 w2 = reinterpret_cast<const uint2*>(row)[g];
        if (sizeof(T) == 2 && wide) {
            uint32_t v[8];
            sm100::unpack16<false>(w2.x, w2.y, row[l.off_scale + g], v);
            uint4* to = reinterpret_cast<uint4*>(dst + g * kPackGroup);
            to[0] = make_uint4(v[0], v[1], v[2], v[3]);
            to[1] = make_uint4(v[4], v[5], v[6], v[7]);
            continue;
        }
        const float s = packed_scale(row[l.off_scale + g]);
        float x[16];
#pragma unroll
        for (int e = 0; e < 16; ++e)
            x[e] = (float)((int)(((e < 8 ? w2.x : w2.y) >> packed_shift(e & 7)) & 15u) - 8) * s;
        if (wide) {
            st16(dst + g * kPackGroup, x);
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) st(dst, g * kPackGroup + e, x[e]);
        }
    }
    const T* k = reinterpret_cast<const T*>(row + l.off_rope);
    for (int e = lane; e < d_r; e += 32) dst[d_c + e] = k[e];
}

// ------------------------------------------------------------------ CUDA-core attention over either kind of row

// Element e of row r of sequence b, as fp32.
template <typename T, bool kPacked>
struct RowReader {
    const uint8_t* base;
    int64_t stride;
    PackedLayout l;
    int d_c;
    __device__ RowReader(const CacheView& c, int b, int d_c_, int d_r) : d_c(d_c_) {
        const int es = kPacked ? 1 : (int)sizeof(T);
        base = static_cast<const uint8_t*>(c.data) + (int64_t)b * c.stride_b * es;
        stride = c.stride_t * es;
        l = packed_layout(d_c, d_r, sizeof(T));
    }
    __device__ const uint8_t* row(int r) const { return base + (int64_t)r * stride; }
    __device__ float at(const uint8_t* row, int e) const {
        if constexpr (kPacked) {
            if (e < d_c) return packed_latent(row, l, e);
            return ld(reinterpret_cast<const T*>(row + l.off_rope), e - d_c);
        } else {
            return ld(reinterpret_cast<const T*>(row), e);
        }
    }
};

constexpr int kAttWarps = 8;
constexpr int kMaxPerLane = 32;  // d_c <= 1024

// One block per (query token, head).  Each warp runs an online softmax over
// rows warp, warp + 8, ...; the eight states are merged at the end.
template <typename T, bool kPacked>
__global__ void __launch_bounds__(kAttWarps * 32)
    attend_rows_kernel(Problem p, const T* __restrict__ q_hat, CacheView cache, const int32_t* __restrict__ seqlens,
                       const int32_t* __restrict__ n_seen, T* __restrict__ o_lat, float* __restrict__ lse, int* status) {
    extern __shared__ float smem[];
    const int row = p.d_c + p.d_r;
    float* sq = smem;            // [row]
    float* sm = sq + row;        // [warps] running maxima
    float* sl = sm + kAttWarps;  // [warps] running sums
    float* so = sl + kAttWarps;  // [warps][d_c]
    const int64_t u = blockIdx.x / p.H;
    const int h = blockIdx.x % p.H;
    const int b = (int)(u / p.q_len), i = (int)(u % p.q_len);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int T_b = seqlens[b];
    T* out = o_lat + ((size_t)u * p.H + h) * p.d_c;
    if (n_seen && i == 0 && h == 0 && threadIdx.x == 0 && n_seen[b] < p.q_len) atomicOr(status, MLA_STATUS_BAD_SEQLEN);
    if (T_b < p.q_len || T_b > cache.T_max) {
        if (threadIdx.x == 0) {
            atomicOr(status, MLA_STATUS_BAD_SEQLEN);
            if (lse) lse[(size_t)u * p.H + h] = -INFINITY;
        }
        for (int c = threadIdx.x; c < p.d_c; c += blockDim.x) st(out, c, 0.f);
        return;
    }
    const int n_keys = T_b - p.q_len + 1 + i;
    const T* q = q_hat + ((size_t)u * p.H + h) * row;
    for (int e = threadIdx.x; e < row; e += blockDim.x) sq[e] = ld(q, e);
    __syncthreads();

    const RowReader<T, kPacked> rd(cache, b, p.d_c, p.d_r);
    float m_run = -INFINITY, l_run = 0.f;
    float acc[kMaxPerLane];
#pragma unroll
    for (int r = 0; r < kMaxPerLane; ++r) acc[r] = 0.f;
    for (int j = warp; j < n_keys; j += kAttWarps) {
        const uint8_t* kr = rd.row(j);
        float s = 0.f;
        for (int e = lane; e < row; e += 32) s = fmaf(sq[e], rd.at(kr, e), s);
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        s *= p.scale;
        // (a score of -infinity has no weight; a NaN one, which fmaxf drops, makes the sums NaN)
        const float m_new = fmaxf(m_run, s), ref = m_new == -INFINITY ? 0.f : m_new;
        const float corr = expf(m_run - ref);
        const float pj = expf(s - ref);
        l_run = l_run * corr + pj;
#pragma unroll
        for (int r = 0; r < kMaxPerLane; ++r) {
            const int c = lane + 32 * r;
            if (c < p.d_c) acc[r] = acc[r] * corr + pj * rd.at(kr, c);
        }
        m_run = m_new;
    }
    if (lane == 0) {
        sm[warp] = m_run;
        sl[warp] = l_run;
    }
#pragma unroll
    for (int r = 0; r < kMaxPerLane; ++r) {
        const int c = lane + 32 * r;
        if (c < p.d_c) so[warp * p.d_c + c] = acc[r];
    }
    __syncthreads();
    float M = -INFINITY;
    for (int w = 0; w < kAttWarps; ++w) M = fmaxf(M, sm[w]);
    float L = 0.f;
    const float ref = M == -INFINITY ? 0.f : M;
    for (int w = 0; w < kAttWarps; ++w) L += sl[w] * expf(sm[w] - ref);
    for (int c = threadIdx.x; c < p.d_c; c += blockDim.x) {
        float o = 0.f;
        for (int w = 0; w < kAttWarps; ++w) o += so[w * p.d_c + c] * expf(sm[w] - ref);
        st(out, c, L == 0.f ? 0.f : o / L);  // (0: every score is -infinity)
    }
    if (lse && threadIdx.x == 0) lse[(size_t)u * p.H + h] = M + logf(L);
}

// A block per eight rows of a sequence, a warp a row: the warp holds the row
// and walks over every query token and head.
template <typename T, bool kPacked>
__global__ void __launch_bounds__(kAttWarps * 32)
    weights_kernel(Problem p, const T* __restrict__ q_hat, const float* __restrict__ lse, CacheView cache,
                   const int32_t* __restrict__ seqlens, float decay, const float* prev, float* weights, int64_t stride_w,
                   int* status) {
    extern __shared__ float smem[];
    const int row = p.d_c + p.d_r;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    float* sk = smem + warp * row;
    for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
        const int T_b = seqlens[b];
        if (T_b < p.q_len || T_b > cache.T_max) {
            if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(status, MLA_STATUS_BAD_SEQLEN);
            continue;
        }
        const RowReader<T, kPacked> rd(cache, b, p.d_c, p.d_r);
        for (int64_t t = (int64_t)blockIdx.x * kAttWarps + warp; t < T_b; t += (int64_t)gridDim.x * kAttWarps) {
            const uint8_t* kr = rd.row((int)t);
            for (int e = lane; e < row; e += 32) sk[e] = rd.at(kr, e);
            __syncwarp();
            float w = 0.f;
            for (int i = 0; i < p.q_len; ++i) {
                if (t > T_b - p.q_len + i) continue;
                for (int h = 0; h < p.H; ++h) {
                    const size_t u = ((size_t)b * p.q_len + i) * p.H + h;
                    const T* q = q_hat + u * row;
                    float s = 0.f;
                    for (int e = lane; e < row; e += 32) s = fmaf(ld(q, e), sk[e], s);
#pragma unroll
                    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                    const float z = lse[u];
                    if (z != -INFINITY) w += expf(s * p.scale - z);
                }
            }
            if (lane == 0) {
                const size_t at = (size_t)b * stride_w + t;
                weights[at] = prev ? fmaf(decay, prev[at], w) : w;
            }
            __syncwarp();
        }
    }
}

template <typename T>
cudaError_t append_t(const Problem& p, bool packed, const void* c_kv, const void* k_rope, const int32_t* pos,
                     const int32_t* rows, int n_tok, const CacheView& cache, int* status, cudaStream_t st) {
    const int64_t tokens = (int64_t)p.B * n_tok;
    const dim3 grid((unsigned)((tokens + kRowWarps - 1) / kRowWarps)), block(kRowWarps * 32);
    if (packed)
        append_packed_kernel<T><<<grid, block, 0, st>>>((const T*)c_kv, (const T*)k_rope, pos, rows, tokens, n_tok, p.d_c,
                                                        p.d_r, cache, p.rope, status);
    else
        append_rows_kernel<T><<<grid, block, 0, st>>>((const T*)c_kv, (const T*)k_rope, pos, rows, tokens, n_tok, p.d_c,
                                                      p.d_r, cache, p.rope, status);
    return cudaGetLastError();
}

template <typename T>
cudaError_t load_t(const Problem& p, const CacheView& cache, const int32_t* rows, int n_tok, void* out, int* status,
                   cudaStream_t st) {
    const int64_t tokens = (int64_t)p.B * n_tok;
    load_packed_kernel<T><<<(unsigned)((tokens + kRowWarps - 1) / kRowWarps), kRowWarps * 32, 0, st>>>(
        cache, rows, tokens, n_tok, p.d_c, p.d_r, (T*)out, status);
    return cudaGetLastError();
}

template <typename T, bool kPacked>
cudaError_t attend_rows_t(const Problem& p, const void* q_hat, const CacheView& cache, const int32_t* seqlens,
                          const int32_t* n_seen, void* o_lat, float* lse, int* status, cudaStream_t st) {
    const size_t smem = sizeof(float) * ((p.d_c + p.d_r) + 2 * kAttWarps + (size_t)kAttWarps * p.d_c);  // at most 38 KB
    attend_rows_kernel<T, kPacked><<<(unsigned)((size_t)p.B * p.q_len * p.H), kAttWarps * 32, smem, st>>>(
        p, (const T*)q_hat, cache, seqlens, n_seen, (T*)o_lat, lse, status);
    return cudaGetLastError();
}

template <typename T, bool kPacked>
cudaError_t weights_t(const Problem& p, const void* q_hat, const float* lse, const CacheView& cache,
                      const int32_t* seqlens, float decay, const float* prev, float* weights, int64_t stride_w,
                      int* status, cudaStream_t st) {
    const size_t smem = sizeof(float) * (size_t)kAttWarps * (p.d_c + p.d_r);  // at most 37 KB
    const int64_t blocks = ((int64_t)cache.T_max + kAttWarps - 1) / kAttWarps;
    weights_kernel<T, kPacked><<<dim3((unsigned)(blocks < 4096 ? blocks : 4096), p.B < 65535 ? p.B : 65535), kAttWarps * 32, smem, st>>>(
        p, (const T*)q_hat, lse, cache, seqlens, decay, prev, weights, stride_w, status);
    return cudaGetLastError();
}

}  // namespace

cudaError_t rows_append(const Problem& p, bool packed, const void* c_kv, const void* k_rope, const int32_t* pos,
                        const int32_t* rows, int n_tok, const CacheView& cache, int* status, cudaStream_t st) {
    return p.dtype == MLA_DTYPE_F32 ? append_t<float>(p, packed, c_kv, k_rope, pos, rows, n_tok, cache, status, st)
                                    : append_t<__nv_bfloat16>(p, packed, c_kv, k_rope, pos, rows, n_tok, cache, status, st);
}

cudaError_t packed_load(const Problem& p, const CacheView& cache, const int32_t* rows, int n_tok, void* out, int* status,
                        cudaStream_t st) {
    return p.dtype == MLA_DTYPE_F32 ? load_t<float>(p, cache, rows, n_tok, out, status, st)
                                    : load_t<__nv_bfloat16>(p, cache, rows, n_tok, out, status, st);
}

cudaError_t generic_attend_rows(const Problem& p, bool packed, const void* q_hat, const CacheView& cache,
                                const int32_t* seqlens, const int32_t* n_seen, void* o_lat, float* lse, int* status,
                                cudaStream_t st) {
#define MLA_ATTEND(T, P) attend_rows_t<T, P>(p, q_hat, cache, seqlens, n_seen, o_lat, lse, status, st)
    if (p.dtype == MLA_DTYPE_F32) return packed ? MLA_ATTEND(float, true) : MLA_ATTEND(float, false);
    return packed ? MLA_ATTEND(__nv_bfloat16, true) : MLA_ATTEND(__nv_bfloat16, false);
#undef MLA_ATTEND
}

cudaError_t generic_weights(const Problem& p, bool packed, const void* q_hat, const float* lse, const CacheView& cache,
                            const int32_t* seqlens, float decay, const float* prev, float* weights, int64_t stride_w,
                            int* status, cudaStream_t st) {
#define MLA_WEIGHTS(T, P) weights_t<T, P>(p, q_hat, lse, cache, seqlens, decay, prev, weights, stride_w, status, st)
    if (p.dtype == MLA_DTYPE_F32) return packed ? MLA_WEIGHTS(float, true) : MLA_WEIGHTS(float, false);
    return packed ? MLA_WEIGHTS(__nv_bfloat16, true) : MLA_WEIGHTS(__nv_bfloat16, false);
#undef MLA_WEIGHTS
}

}  // namespace mla
