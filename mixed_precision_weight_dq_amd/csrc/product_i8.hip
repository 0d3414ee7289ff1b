// Integer products of int8 activations (tokens.hip) and packed b-bit weights,
// 2 <= b <= 8:
//   y[m,n] = sx[m] * sw[n] * sum_k xq[m,k] (u[n,k] - z[n]),
// u the stored codes, z = 2^(b-1) (symmetric) or the row's zero point.  The sum
// is exact: with c = 128 for b = 8 (u xor 0x80 is u - 128 as a signed byte) and
// c = 0 below (u < 128 is a signed byte as it is), the matrix cores add
// xq * (u - c) in int32, and (z - c) * sum_k xq comes off in the epilogue.
// |xq| <= 128, |u - z| <= 255 and K <= 65536 keep every sum inside int32.
// Three roundings follow: the sum to fp32, times sx, times sw (and one more to
// bf16 when y is bf16).
#include "common.hpp"
#include "i8_tiles.hpp"
#include "launch_serving.hpp"

namespace dq {

namespace {

constexpr int kBM = 64;
constexpr int kBN = 64;
constexpr int kBK = 128;
constexpr int kLd = kBK + 16;  // LDS row pitch in bytes
constexpr int kThreads = 256;

template <int B, bool kBf16Out>
__global__ __launch_bounds__(kThreads) void gemm_i8_kernel(
    const int8_t* __restrict__ x, const float* __restrict__ x_scales,
    const int32_t* __restrict__ x_sums, int64_t M, int64_t pitch,
    const uint32_t* __restrict__ packed, const float* __restrict__ scales,
    const int32_t* __restrict__ zeros, int64_t N, int64_t row_words, void* __restrict__ y)
{
    __shared__ __attribute__((aligned(16))) int8_t As[kBM * kLd];
    __shared__ __attribute__((aligned(16))) int8_t Bs[kBN * kLd];
    const int tid = threadIdx.x;
    const int lane = tid & (kWave - 1);
    const int wave = tid / kWave;
    const int64_t ntn = ceil_div(N, kBN);
    const int64_t m0 = (blockIdx.x / ntn) * kBM;
    const int64_t n0 = (blockIdx.x % ntn) * kBN;
    const int sr = tid >> 2;  // staging row
    const int sc = tid & 3;   // staging chunk of 32
    i32x4_t acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = (i32x4_t){0, 0, 0, 0};

    for (int64_t k0 = 0; k0 < pitch; k0 += kBK) {
        uint4 a[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if (m0 + sr < M) {
            const uint4* src = reinterpret_cast<const uint4*>(x + (m0 + sr) * pitch + k0 + 32 * sc);
            a[0] = src[0];
            a[1] = src[1];
        }
        uint32_t w[B];
        const int64_t n = n0 + sr < N ? n0 + sr : N - 1;
        load_chunk_words<B>(packed + n * row_words, k0 / kChunk + sc, row_words, w);
        i32x4_t b0 = expand16<B>(w, 0), b1 = expand16<B>(w, 1);
        uint4* da = reinterpret_cast<uint4*>(As + sr * kLd + 32 * sc);
        da[0] = a[0];
        da[1] = a[1];
        i32x4_t* db = reinterpret_cast<i32x4_t*>(Bs + sr * kLd + 32 * sc);
        db[0] = b0;
        db[1] = b1;
        __syncthreads();
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int col = 64 * t + 16 * (lane >> 4);
            const i32x4_t av = *reinterpret_cast<const i32x4_t*>(As + (wave * 16 + (lane & 15)) * kLd + col);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const i32x4_t bv = *reinterpret_cast<const i32x4_t*>(Bs + (j * 16 + (lane & 15)) * kLd + col);
                acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(av, bv, acc[j], 0, 0, 0);
            }
        }
        __syncthreads();
    }
    // lane holds column lane & 15, rows 4 (lane >> 4) + r
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t n = n0 + j * 16 + (lane & 15);
        if (n >= N) continue;
        const float sw = scales[n];
        const int32_t z = code_shift<B>(zeros, n);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int64_t m = m0 + wave * 16 + 4 * (lane >> 4) + r;
            if (m < M)
                store_y<kBf16Out>(y, m * N + n, finish_i8(acc[j][r], z, x_sums[m], x_scales[m], sw));
        }
    }
}

template <int B>
hipError_t launch_b(const int8_t* x, const float* xs, const int32_t* xsum, int64_t M,
                    const uint32_t* packed, const float* scales, const int32_t* zeros, int64_t N,
                    int64_t K, void* y, bool bf16, hipStream_t stream)
{
    const int64_t pitch = token_row_bytes(K), rw = packed_row_words(K, B);
    const int64_t tiles = ceil_div(M, kBM) * ceil_div(N, kBN);
    if (tiles > 0x7fffffffLL) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)tiles);
    if (bf16)
        gemm_i8_kernel<B, true><<<grid, kThreads, 0, stream>>>(x, xs, xsum, M, pitch, packed, scales,
                                                              zeros, N, rw, y);
    else
        gemm_i8_kernel<B, false><<<grid, kThreads, 0, stream>>>(x, xs, xsum, M, pitch, packed, scales,
                                                               zeros, N, rw, y);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_i8(const int8_t* x, const float* x_scales, const int32_t* x_sums, int64_t M,
                          const uint32_t* packed, const float* scales, const int32_t* zeros,
                          int64_t N, int64_t K, int bits, void* y, bool bf16, hipStream_t stream)
{
#define CALL(B) launch_b<B>(x, x_scales, x_sums, M, packed, scales, zeros, N, K, y, bf16, stream)
    DQ_I8_BITS_SWITCH(bits, CALL)
#undef CALL
}

}  // namespace dq
