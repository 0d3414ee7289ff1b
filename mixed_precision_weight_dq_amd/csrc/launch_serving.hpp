// Host-side launchers of the int8 activation and 4-bit cache kernels (internal,
// as launch.hpp: arguments are validated by the caller).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cache4.hpp"
#include "layout.hpp"
#include "rope.hpp"

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
// the same, keys rotated at positions[token] (null: their positions in the sequences)
hipError_t launch_cache4_append_rope(const Cache4& c, const Cache4Batch& bt, const void* k, const void* v,
                                     bool bf16, int64_t tokens, int64_t k_stride, int64_t v_stride,
                                     const Rope& rope, const int32_t* positions, hipStream_t stream);
// new row path[first + j] of each sequence -> row j, j < accepted[b]
hipError_t launch_cache4_keep(const Cache4& c, const Cache4Batch& bt, const int32_t* path,
                              const int32_t* accepted, int64_t tokens, hipStream_t stream);
hipError_t launch_cache4_read(const Cache4& c, const Cache4Batch& bt, void* k, void* v, bool bf16,
                              int64_t tokens, hipStream_t stream);
hipError_t launch_cache4_attention(const Cache4& c, const Cache4Batch& bt, const uint16_t* q,
                                   int64_t tokens, int64_t q_stride, int q_heads, float scale,
                                   int64_t max_q, int64_t max_len, uint16_t* out, void* workspace,
                                   hipStream_t stream);
// Bytes of `workspace` that launch_cache4_attention uses for these arguments (0: none).
size_t cache4_attention_workspace(const Cache4& c, int64_t count, int64_t tokens,
                                  int q_heads, int64_t max_q, int64_t max_len);

// mask: bit j of a token's `words` words: it sees its sequence's new token j
hipError_t launch_cache4_tree(const Cache4& c, const Cache4Batch& bt, const uint16_t* q, int64_t tokens,
                              int64_t q_stride, int q_heads, const int32_t* mask, int64_t words,
                              float scale, int64_t max_q, int64_t max_len, uint16_t* out,
                              void* workspace, hipStream_t stream);
size_t cache4_tree_workspace(const Cache4& c, int64_t count, int64_t tokens, int q_heads, int64_t max_q,
                             int64_t max_len);

// out = x with its first rope.dims dimensions rotated; strides in elements
hipError_t launch_rotate(const Rope& rope, const void* x, bool bf16, int64_t tokens, int heads, int dim,
                         int64_t x_token, int64_t x_head, const int32_t* positions, void* out,
                         int64_t out_token, int64_t out_head, hipStream_t stream);

// Rows of a sequence that its tree can have.  Looking for ids that came before takes a pass over the rows
// for each candidate, some 60 ms where all of these are one row's children: without a limit a call could
// run for minutes.
constexpr int64_t kMaxDrafts = 4096;

struct VerifyArgs {
    const float* probs;  // [tokens, vocab], rows probs_stride apart
    int64_t probs_stride;
    const float* draft;  // nullptr, or the same of the drafts
    int64_t draft_stride;
    const int32_t* ids;
    const int32_t* parents;
    const int32_t* starts;
    const float* uniforms;
    int64_t tokens, count, vocab;
    int32_t* path;      // [tokens]
    int32_t* accepted;  // [count]
    int32_t* next;      // [count]
    double* sums;       // set by launch_verify, in the workspace: [count, chunks]
    int64_t chunks;
    int32_t* state;     // [count, 2]: last row taken, whether draft probabilities come off
};
hipError_t launch_verify(VerifyArgs a, void* workspace, hipStream_t stream);
size_t verify_workspace(int64_t count, int64_t vocab);
hipError_t launch_draft_tree(const int32_t* parents, const int32_t* starts, const int32_t* lens, int64_t count,
                             int64_t tokens, int64_t words, int32_t* mask, int32_t* positions, hipStream_t stream);

}  // namespace dq
