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
// (two of fp32) and one 8-byte store of codes.  A thread keeps its first kHeld
// pieces (rows of up to 8192 elements whole) in registers between the maximum and
// the codes; of longer rows the rest is read again, from the caches by then.  Bound
// by memory: 2048 x 8192 in bf16 (34 MB in, 17 MB out) 11.8 us, 4.3 TB/s (every row
// read twice: 15.5 us); 1 x 4096 3.3 us, a launch and two trips to memory.
#include "common.hpp"
#include "launch_serving.hpp"
#include "quant_rule.hpp"

namespace dq {

namespace {

constexpr int kPiece = 8;
constexpr int kTokenThreads = 256;
constexpr int kHeld = 4;  // pieces per thread
constexpr int64_t kLaunchTokens = 1LL << 23;  // (a multiple of 16 bytes of x for any K)

// The 8 elements of a piece as they lie in memory.
template <bool BF16>
struct Piece {
    uint32_t w[BF16 ? 4 : 8];
    __device__ __forceinline__ void floats(float (&v)[kPiece]) const
    {
#pragma unroll
        for (int e = 0; e < kPiece; ++e)
            v[e] = __uint_as_float(!BF16 ? w[BF16 ? 0 : e] : (e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16));
    }
};

// Piece p of a row, 0 past its end.
template <bool BF16>
__device__ __forceinline__ Piece<BF16> load_piece(const void* __restrict__ x, int64_t row_off,
                                                  int64_t K, int64_t p, bool vec)
{
    Piece<BF16> d;
    const int64_t k0 = p * kPiece;
    if (vec && k0 + kPiece <= K) {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const char*>(x) +
                                                          (row_off + k0) * (BF16 ? 2 : 4));
#pragma unroll
        for (int h = 0; h < (BF16 ? 1 : 2); ++h) {
            const uint4 a = src[h];
            d.w[4 * h] = a.x, d.w[4 * h + 1] = a.y, d.w[4 * h + 2] = a.z, d.w[4 * h + 3] = a.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < (BF16 ? 4 : 8); ++i) {
            if (BF16) {
                const uint16_t* src = static_cast<const uint16_t*>(x) + row_off + k0 + 2 * i;
                d.w[i] = (k0 + 2 * i < K ? (uint32_t)src[0] : 0u) |
                         (k0 + 2 * i + 1 < K ? (uint32_t)src[1] << 16 : 0u);
            } else {
                d.w[i] = k0 + i < K ? static_cast<const uint32_t*>(x)[row_off + k0 + i] : 0u;
            }
        }
    }
    return d;
}

template <bool BF16>
__device__ __forceinline__ uint32_t piece_max(const Piece<BF16>& d, uint32_t amax)
{
    float v[kPiece];
    d.floats(v);
#pragma unroll
    for (int e = 0; e < kPiece; ++e) amax = max(amax, __float_as_uint(v[e]) & 0x7fffffffu);
    return amax;
}

// A piece's codes and their sum.
template <bool BF16>
__device__ __forceinline__ uint2 piece_codes(const Piece<BF16>& d, float s, float r, bool zero, int& sum)
{
    float v[kPiece], q[kPiece];
    d.floats(v);
    clipped_quotients(v, s, r, quotient_margin(128.0f), 127.0f, q);
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        // two codes at a time as the exact fp32 value (q0 + 128) + 256 (q1 + 128)
        const float lo = fmaf(q[4 * h + 1], 256.0f, q[4 * h] + 32896.0f);
        const float hi = fmaf(q[4 * h + 3], 256.0f, q[4 * h + 2] + 32896.0f);
        w[h] = zero ? 0u : ((uint32_t)hi << 16 | (uint32_t)lo) ^ 0x80808080u;
        sum = __builtin_amdgcn_sdot4((int)w[h], 0x01010101, sum, false);
    }
    return make_uint2(w[0], w[1]);
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

    // max |x| as an integer max over sign-cleared bit patterns
    Piece<BF16> held[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
        if (tid + i * kTokenThreads < pieces)
            held[i] = load_piece<BF16>(x, row_off, K, tid + i * kTokenThreads, vec);
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
        if (tid + i * kTokenThreads < pieces) amax = piece_max<BF16>(held[i], amax);
    for (int64_t p = tid + kHeld * kTokenThreads; p < pieces; p += kTokenThreads)
        amax = piece_max<BF16>(load_piece<BF16>(x, row_off, K, p, vec), amax);
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

    // codes and their sum (elements past K are 0, so is their code)
    int32_t sum = 0;
    uint2* out = reinterpret_cast<uint2*>(codes + m * pitch);
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
        if (tid + i * kTokenThreads < pieces)
            out[tid + i * kTokenThreads] = piece_codes<BF16>(held[i], s, r, zero_codes, sum);
    for (int64_t p = tid + kHeld * kTokenThreads; p < pieces; p += kTokenThreads)
        out[p] = piece_codes<BF16>(load_piece<BF16>(x, row_off, K, p, vec), s, r, zero_codes, sum);
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
    // a launch has at most 2^32 - 1 threads
    for (int64_t m = 0; m < M; m += kLaunchTokens) {
        const dim3 grid((unsigned)(M - m < kLaunchTokens ? M - m : kLaunchTokens));
        const void* row = static_cast<const char*>(x) + m * K * (bf16 ? 2 : 4);
        (bf16 ? quantize_tokens_kernel<true> : quantize_tokens_kernel<false>)<<<grid, kTokenThreads, 0, stream>>>(
            row, K, pitch, codes + m * pitch, scales + m, sums + m);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace dq
