// Host-side launchers of the int8 activation and 4-bit cache kernels (internal,
// as launch.hpp: arguments are validated by the caller).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cache4.hpp"
#include "layout.hpp"

namespace dq {

// codes [M, token_row_bytes(K)], scales and code sums [M] of the tokens of x
hipError_t launch_quantize_tokens(const void* x, bool bf16, int64_t M, int64_t K, int8_t* codes,
                                  float* scales, int32_t* sums, hipStream_t stream);
// y[m, n] = x_scales[m] * scales[n] * sum_k x[m, k] (u[n, k] - z[n]), bits <= 8;
// zeros as for launch_gemv, y fp32 or bf16
hipError_t launch_gemm_i8(const int8_t* x, const float* x_scales, const int32_t* x_sums, int64_t M,
                          const uint32_t* packed, const float* scales, const int32_t* zeros,
                          int64_t N, int64_t K, int bits, void* y, bool bf16, hipStream_t stream);

hipError_t launch_cache4_append(const Cache4& c, const Cache4Batch& bt, const void* k,
                                const void* v, bool bf16, int64_t tokens, int64_t k_stride,
                                int64_t v_stride, hipStream_t stream);
hipError_t launch_cache4_read(const Cache4& c, const Cache4Batch& bt, void* k, void* v, bool bf16,
                              int64_t tokens, hipStream_t stream);
hipError_t launch_cache4_attention(const Cache4& c, const Cache4Batch& bt, const uint16_t* q,
                                   int64_t tokens, int64_t q_stride, int q_heads, float scale,
                                   int64_t max_q, int64_t max_len, uint16_t* out, void* workspace,
                                   hipStream_t stream);
// Bytes of `workspace` that launch_cache4_attention uses for these arguments (0: none).
size_t cache4_attention_workspace(const Cache4& c, int64_t count, int64_t tokens,
                                  int q_heads, int64_t max_q, int64_t max_len);

}  // namespace dq
