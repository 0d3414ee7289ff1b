// Per-token int8 activations: the symmetric rule of the "量化" tutorial
// (aiknowledge.cn), "how quantization works", at b = 8 with one token (row of
// x) as the channel:
//   s[m] = fl32(max_k |x[m,k]| / 127)  (1.0 replaces a zero max),
//   q[m,k] = clip(rint(fl32(x[m,k] / s[m])), -128, 127)
// in IEEE fp32, so a token's codes are those of dq_quantize_pack at b = 8 as
// signed bytes.  Beside them goes sum_k q[m,k] (int32), which takes the weight
// codes' offset or zero point off an integer product exactly.
//
// One workgroup per token.  A piece is 8 elements: one 16-byte load of bf16
// (two of fp32) and one 8-byte store of codes.
#include "common.hpp"
#include "launch_serving.hpp"
#include "quant_rule.hpp"

namespace dq {

namespace {

constexpr int kPiece = 8;
constexpr int kTokenThreads = 256;

// The 8 elements of piece p of a row, 0 past its end.
template <bool BF16>
__device__ __forceinline__ void load_piece(const void* __restrict__ x, int64_t row_off, int64_t K,
                                           int64_t p, bool vec, float (&v)[kPiece])
{
    const int64_t k0 = p * kPiece;
    if (vec && k0 + kPiece <= K) {
        if (BF16) {
            const uint4 d = *reinterpret_cast<const uint4*>(
                static_cast<const uint16_t*>(x) + row_off + k0);
            const uint32_t u[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[2 * e] = __uint_as_float(u[e] << 16);
                v[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
            }
        } else {
            const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(x) + row_off + k0);
            const float4 a = q[0], b = q[1];
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
            v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < kPiece; ++e) {
            if (k0 + e >= K)
                v[e] = 0.0f;
            else
                v[e] = BF16 ? bf16_bits_to_float(static_cast<const uint16_t*>(x)[row_off + k0 + e])
                            : static_cast<const float*>(x)[row_off + k0 + e];
        }
    }
}

template <bool BF16>
__global__ __launch_bounds__(kTokenThreads) void quantize_tokens_kernel(
    const void* __restrict__ x, int64_t K, int64_t pitch, int8_t* __restrict__ codes,
    float* __restrict__ scales, int32_t* __restrict__ sums)
{
    constexpr int kWaves = kTokenThreads / kWave;
    __shared__ uint32_t red_max[kWaves];
    __shared__ int32_t red_sum[kWaves];
    const int64_t m = blockIdx.x;
    const int tid = threadIdx.x;
    const int64_t row_off = m * K;
    const int64_t pieces = pitch / kPiece;
    const bool vec = (K * (BF16 ? 2 : 4)) % 16 == 0;

    // pass 1: max |x| as an integer max over sign-cleared bit patterns
    uint32_t amax = 0;
    for (int64_t p = tid; p < pieces; p += kTokenThreads) {
        float v[kPiece];
        load_piece<BF16>(x, row_off, K, p, vec, v);
#pragma unroll
        for (int e = 0; e < kPiece; ++e) {
            const uint32_t a = __float_as_uint(v[e]) & 0x7fffffffu;
            amax = a > amax ? a : amax;
        }
    }
    amax = wave_max_u32(amax);
    if ((tid & (kWave - 1)) == 0) red_max[tid / kWave] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWaves; ++i) amax = red_max[i] > amax ? red_max[i] : amax;

    float s;
    bool zero_codes = false;
    if (amax >= 0x7f800000u) {  // a NaN or an infinity in the token
        s = __uint_as_float(0x7fc00000u);
        zero_codes = true;
    } else {
        const float a = __uint_as_float(amax);
        s = (a == 0.0f ? 1.0f : a) / 127.0f;
        if (a == 0.0f || s == 0.0f) {  // all zero, or a max whose quotient underflows
            s = 1.0f / 127.0f;
            zero_codes = true;
        }
    }
    const float r = 1.0f / s;
    const float margin = quotient_margin(128.0f);

    // pass 2: codes and their sum (elements past K are 0, so is their code)
    int32_t sum = 0;
    for (int64_t p = tid; p < pieces; p += kTokenThreads) {
        float v[kPiece];
        load_piece<BF16>(x, row_off, K, p, vec, v);
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int e = 0; e < kPiece; ++e) {
            const float q = fminf(fmaxf(rounded_quotient(v[e], s, r, margin), -128.0f), 127.0f);
            const int32_t c = zero_codes ? 0 : (int32_t)q;
            sum += c;
            w[e >> 2] |= (uint32_t)(c & 0xff) << (8 * (e & 3));
        }
        *reinterpret_cast<uint2*>(codes + m * pitch + p * kPiece) = make_uint2(w[0], w[1]);
    }
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1) sum += __shfl_xor(sum, o, kWave);
    if ((tid & (kWave - 1)) == 0) red_sum[tid / kWave] = sum;
    __syncthreads();
    if (tid == 0) {
        int32_t t = 0;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) t += red_sum[i];
        scales[m] = s;
        sums[m] = t;
    }
}

}  // namespace

hipError_t launch_quantize_tokens(const void* x, bool bf16, int64_t M, int64_t K, int8_t* codes,
                                  float* scales, int32_t* sums, hipStream_t stream)
{
    const int64_t pitch = token_row_bytes(K);
    const dim3 grid((unsigned)M);
    if (bf16)
        quantize_tokens_kernel<true><<<grid, kTokenThreads, 0, stream>>>(x, K, pitch, codes, scales, sums);
    else
        quantize_tokens_kernel<false><<<grid, kTokenThreads, 0, stream>>>(x, K, pitch, codes, scales, sums);
    return hipGetLastError();
}

}  // namespace dq
