// Code expansion and epilogue of the int8 products: 16 consecutive codes of a
// chunk (32 codes in B whole words) as 16 signed bytes of an integer matrix
// operand.  For B <= 7 the bytes are the stored codes u (below 128, so signed
// bytes as they are); for B = 8 they are u - 128.
#pragma once

#include "common.hpp"

namespace dq {

typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));
typedef int32_t i32x16_t __attribute__((ext_vector_type(16)));

// Four B-bit codes in the low 4B bits of v (higher bits may be set) -> bytes.
template <int B>
__device__ __forceinline__ uint32_t spread4(uint32_t v)
{
    // pairs of codes to the two halves, then single codes to the bytes
    constexpr uint32_t kPair = (1u << (2 * B)) - 1u;
    constexpr uint32_t kCode = (1u << B) - 1u;
    const uint32_t t = (v & kPair) | ((v << (16 - 2 * B)) & (kPair << 16));
    return (t & (kCode * 0x00010001u)) | ((t << (8 - B)) & (kCode * 0x01000100u));
}

// Codes 16t .. 16t+15 (t = 0, 1) of a chunk (raw words w).
template <int B>
__device__ __forceinline__ i32x4_t expand16(const uint32_t (&w)[B], int t)
{
    i32x4_t r;
    if constexpr (B == 8) {
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = (int32_t)(w[4 * t + j] ^ 0x80808080u);
    } else if constexpr (B == 4) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t v = w[2 * t + j];
            const uint32_t ev = v & 0x0f0f0f0fu, od = (v >> 4) & 0x0f0f0f0fu;
            r[2 * j] = (int32_t)__builtin_amdgcn_perm(od, ev, 0x05010400u);
            r[2 * j + 1] = (int32_t)__builtin_amdgcn_perm(od, ev, 0x07030602u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int pos = (16 * t + 4 * j) * B;
            const int wi = pos >> 5, off = pos & 31;
            const uint32_t v = off + 4 * B <= 32 ? w[wi] >> off
                                                 : __builtin_amdgcn_alignbit(w[wi + 1 < B ? wi + 1 : wi], w[wi], off);
            r[j] = (int32_t)spread4<B>(v);
        }
    }
    return r;
}

// What the epilogue takes off per unit of the token's code sum: z - c, with z
// the row's zero point (2^(B-1) without zeros) and c = 128 for B = 8, else 0.
template <int B>
__device__ __forceinline__ int32_t code_shift(const int32_t* __restrict__ zeros, int64_t n)
{
    return (zeros ? zeros[n] : (1 << (B - 1))) - (B == 8 ? 128 : 0);
}

// A token's scale as two factors: the sum (below 2^31) times the scale itself would
// pass fp32 from 2^97 on, where the weights' scale may bring the product back.
struct TokenScale {
    float s, up;
};
__device__ __forceinline__ TokenScale token_scale(float sx)
{
    return sx >= 0x1p96f ? TokenScale{sx * 0x1p-32f, 0x1p32f} : TokenScale{sx, 1.0f};
}

// acc - shift * sum is exact (unsigned arithmetic wraps; the result fits), so is
// the last factor.
__device__ __forceinline__ float finish_i8(int32_t acc, int32_t shift, int32_t sum, TokenScale sx, float sw)
{
    const int32_t d = (int32_t)((uint32_t)acc - (uint32_t)shift * (uint32_t)sum);
    return ((float)d * sx.s) * sw * sx.up;
}

__device__ __forceinline__ uint16_t bf16_round(float v)
{
    return __builtin_bit_cast(uint16_t, (__bf16)v);
}

template <bool kBf16>
__device__ __forceinline__ void store_y(void* __restrict__ y, int64_t i, float v)
{
    if constexpr (kBf16)
        static_cast<uint16_t*>(y)[i] = bf16_round(v);
    else
        static_cast<float*>(y)[i] = v;
}

// Expands CALL(B) for the widths an int8 operand holds.
#define DQ_I8_BITS_SWITCH(bits, CALL)                                                             \
    switch (bits) {                                                                               \
    case 2: return CALL(2);                                                                       \
    case 3: return CALL(3);                                                                       \
    case 4: return CALL(4);                                                                       \
    case 5: return CALL(5);                                                                       \
    case 6: return CALL(6);                                                                       \
    case 7: return CALL(7);                                                                       \
    case 8: return CALL(8);                                                                       \
    default: return hipErrorInvalidValue;                                                         \
    }

}  // namespace dq
