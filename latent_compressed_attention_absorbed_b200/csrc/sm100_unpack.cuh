// Packed 4-bit rows in registers: sixteen latents of a group as eight pairs of
// bf16 or fp16 values, exactly (the format is described in mla_packed.cuh).
#pragma once

#include <stdint.h>

#include "mla_packed.cuh"
#include "sm100_ptx.cuh"

namespace mla {
namespace sm100 {

constexpr int kPackNib = 256;    // bytes of codes of a V3 row
constexpr int kPackScale = 32;   // bytes of scales
constexpr int kPackRope = 288;   // where its key starts

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Pairs 0..7 of a group from its two words and its scale byte, with the fewest
// instructions, as the kernels that unpack are bound by their number: a code
// under a suitable exponent reads as a number, and one fused multiply-add with
// the scale takes its offset off, exactly.
//   bf16: under the exponent of 128 the lowest four fraction bits read 128 + n,
//         and (128 + n) s - 136 s = q s (136 s has eight significant bits); the
//         first pair needs no shift, and a scale byte becomes a pair of bf16
//         scales by one integer multiply-add;
//   fp16: under the exponent of 16 the four leading fraction bits read 16 + n,
//         and (16 + n) s - 24 s = q s (136 s would pass the largest fp16).
template <bool kF16>
__device__ __forceinline__ void unpack16(uint32_t w0, uint32_t w1, uint32_t scale_byte, uint32_t (&out)[8]) {
    if constexpr (kF16) {
        const float s = packed_scale(scale_byte);
        const uint32_t s2 = pack_f16(s, s), c2 = mul_f16x2(s2, 0xCE00CE00u);  // -24
        constexpr uint32_t kMask = 0x03C003C0u, kOne = 0x4C004C00u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t w = h ? w1 : w0;
            out[4 * h + 0] = fma_f16x2(((w << 6) & kMask) | kOne, s2, c2);
            out[4 * h + 1] = fma_f16x2(((w << 2) & kMask) | kOne, s2, c2);
            out[4 * h + 2] = fma_f16x2(((w >> 2) & kMask) | kOne, s2, c2);
            out[4 * h + 3] = fma_f16x2(((w >> 6) & kMask) | kOne, s2, c2);
        }
    } else {
        const uint32_t s2 = scale_byte * 0x00100010u + ((127u - kPackScaleBias) << 7) * 0x00010001u;
        const uint32_t c2 = mul_bf16x2(s2, 0xC308C308u);  // -136
        constexpr uint32_t kMask = 0x000F000Fu, kOne = 0x43004300u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t w = h ? w1 : w0;
            out[4 * h + 0] = fma_bf16x2((w & kMask) | kOne, s2, c2);
            out[4 * h + 1] = fma_bf16x2(((w >> 4) & kMask) | kOne, s2, c2);
            out[4 * h + 2] = fma_bf16x2(((w >> 8) & kMask) | kOne, s2, c2);
            out[4 * h + 3] = fma_bf16x2(((w >> 12) & kMask) | kOne, s2, c2);
        }
    }
}

// The codes and scales of 64 latents (chunk c) of a raw row in shared memory.
struct RawChunk {
    uint32_t w[8], scales;
    __device__ __forceinline__ void load(uint32_t raw_row, int c) {
        scales = ld_shared_u32(raw_row + kPackNib + 4 * c);
        ld_shared_v4u(raw_row + 32 * c, w[0], w[1], w[2], w[3]);
        ld_shared_v4u(raw_row + 32 * c + 16, w[4], w[5], w[6], w[7]);
    }
    // The same by loads that the compiler keeps where they stand and does once.
    __device__ __forceinline__ void load_once(uint32_t raw_row, int c) {
        asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(scales) : "r"(raw_row + kPackNib + 4 * c) : "memory");
#pragma unroll
        for (int h = 0; h < 2; ++h)
            asm volatile("ld.volatile.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[4 * h]), "=r"(w[4 * h + 1]), "=r"(w[4 * h + 2]), "=r"(w[4 * h + 3])
                         : "r"(raw_row + 32 * c + 16 * h)
                         : "memory");
    }
    // -> 128 bytes of values at row `row` of a swizzled chunk of 128-byte rows.
    // at: the row's first piece, chunk + 128 row + 16 (row % 8); piece j lies at
    // at ^ 16 j (the chunk starts on a 1024-byte boundary).
    template <bool kF16>
    __device__ __forceinline__ void unpack(uint32_t at) const {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            uint32_t v[8];
            unpack16<kF16>(w[2 * g], w[2 * g + 1], (scales >> (8 * g)) & 0xFFu, v);
            st_shared_v4(at ^ (32 * g), v[0], v[1], v[2], v[3]);
            st_shared_v4(at ^ (32 * g + 16), v[4], v[5], v[6], v[7]);
        }
    }
};

}  // namespace sm100
}  // namespace mla
