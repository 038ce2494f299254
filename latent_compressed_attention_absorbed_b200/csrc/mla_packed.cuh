// The 4-bit cache row and its arithmetic, shared by every kernel that writes
// or reads packed rows.
//
// A packed row holds the d_c latents of a token in 4 bits each, one 8-bit
// scale for every 16 of them, and the rotated RoPE key unquantised (a key's
// error would move every score of its row, and it is a ninth of the values):
//   bytes [0, d_c/2)               codes n = q + 8, q in -7..7: element 8w + 2j of 32-bit word w in bits 4j..4j+3,
//                                  element 8w + 2j + 1 in bits 16+4j..19+4j
//   bytes [d_c/2, d_c/2 + d_c/16)  scales, e * 8 + m standing for 2^(e-21) (1 + m/8)
//   from there, rounded up to 16   the RoPE key in the cache's type; the row ends on a multiple of 16 bytes
// 416 bytes for d_c = 512 and a 64-wide bf16 key.
//
// A uniform grid of 15 levels has a smaller rms error on normally distributed
// groups of 16 than a 4-bit floating-point grid of the same range (0.085 of
// the rms against 0.095), and it unpacks with one fused multiply-add for two
// values, exactly.  The scale has four significant bits
// (3 stored), five exponent bits and no zero, infinity or NaN, so whatever
// bytes a row holds, the latents it stands for are finite numbers; every
// value q s is exact in bf16 and, as a multiple of 2^-24 below 2^14, in fp16.
// The scale of a group is the smallest that is not below max|x| / 7: nothing
// is clipped up to |x| = 13440, and x is rounded to the nearest multiple,
// half to even.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace mla {

constexpr int kPackGroup = 16;      // latents that share a scale
constexpr int kPackScaleBias = 21;  // exponent bias of a scale

struct PackedLayout {
    int off_scale, off_rope, bytes;
};
__host__ __device__ inline PackedLayout packed_layout(int d_c, int d_r, int elem) {
    PackedLayout l;
    l.off_scale = d_c / 2;
    l.off_rope = (d_c / 2 + d_c / kPackGroup + 15) & ~15;
    l.bytes = (l.off_rope + d_r * elem + 15) & ~15;
    return l;
}

// The number a scale byte stands for.
__device__ __forceinline__ float packed_scale(uint32_t code) {
    return __uint_as_float((code << 20) + ((127u - kPackScaleBias) << 23));
}

// The smallest scale s with 7 s >= amax (255 if there is none); amax finite and not negative.
__device__ __forceinline__ uint32_t packed_scale_code(float amax) {
    // the quotient's three leading fraction bits, rounded up, then put right
    // against the exact products 7 s (seven significant bits)
    const int bits = (int)((__float_as_uint(amax * (1.0f / 7.0f)) + 0xFFFFFu) >> 20) - ((127 - kPackScaleBias) << 3);
    int c = bits < 0 ? 0 : (bits > 255 ? 255 : bits);
    if (c < 255 && 7.0f * packed_scale(c) < amax) ++c;
    if (c > 0 && 7.0f * packed_scale(c - 1) >= amax) --c;
    return (uint32_t)c;
}

// Nearest integer to x / s, half to even, clipped to -7..7.  The product with
// the rounded reciprocal may fall on the wrong side of a half; x - q s is
// exact (q s is close to x), so the side is decided by it.
__device__ __forceinline__ int packed_quantise(float x, float s, float inv_s) {
    float q = rintf(x * inv_s);
    q = fminf(fmaxf(q, -7.0f), 7.0f);
    const float r = fmaf(-q, s, x);
    const float twice = 2.0f * fabsf(r);
    if (twice > s || (twice == s && ((int)q & 1))) q += r > 0.0f ? 1.0f : -1.0f;
    return (int)fminf(fmaxf(q, -7.0f), 7.0f);
}

// The same for x with eight significant bits (a bf16 value), as q + 8 in the
// low four bits.  Where |x / s| is at least 0.4, x / s is a multiple of 2^-7 / S
// with S the scale's four bits, so it is either exactly a half or at least
// 5e-4 away from one: rounded to a multiple of 2^-13 (the unit in the last
// place at 1536) the product with the rounded reciprocal falls on a half
// exactly where x / s does, and the addition then rounds halves to even.
__device__ __forceinline__ uint32_t packed_code_bf16(float x, float inv_s) {
    const float snapped = fmaf(x, inv_s, 1536.0f);
    return __float_as_uint(snapped + (12582912.0f + 8.0f - 1536.0f)) & 15u;  // 1.5 * 2^23: the unit in the last place is 1
}

// Word bit position of element e (0..7) of a word.
__host__ __device__ constexpr int packed_shift(int e) { return 4 * (e >> 1) + 16 * (e & 1); }

// One packed latent.
__device__ __forceinline__ float packed_latent(const uint8_t* row, const PackedLayout& l, int c) {
    const uint32_t w = reinterpret_cast<const uint32_t*>(row)[c >> 3];
    const int q = (int)((w >> packed_shift(c & 7)) & 15u) - 8;
    return (float)q * packed_scale(row[l.off_scale + c / kPackGroup]);
}

}  // namespace mla
