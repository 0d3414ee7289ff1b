// C ABI of the library (declared in include/dq.h): argument validation on the
// host, then the kernel launches on the caller's stream.  No allocation, no
// synchronisation, no state beyond the per-thread text of the last HIP error.
// (The host-only allocation entry points live in recipe.cpp, the file format's
// writer and parser in packfile.cpp.)
#include "../../include/dq.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdio>
#include <cstring>

#include "launch.hpp"
#include "launch_serving.hpp"

namespace {

thread_local char g_last_error[256] = "";

dq_status hip_status(hipError_t e)
{
    if (e == hipSuccess) return DQ_OK;
    std::snprintf(g_last_error, sizeof g_last_error, "%s: %s", hipGetErrorName(e),
                  hipGetErrorString(e));
    return DQ_ERR_HIP;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

dq_status check_common(int64_t N, int64_t K, int32_t bits)
{
    if (bits < DQ_MIN_BITS || bits > DQ_MAX_BITS) return DQ_ERR_BITS;
    if (N < 1 || N > 0x7fffffffLL || K < 1 || K > DQ_MAX_K) return DQ_ERR_SHAPE;
    return DQ_OK;
}

// group sizes: powers of two from one chunk (32 codes) to 2048
bool valid_group(int64_t g) { return g >= 32 && g <= DQ_MAX_GROUP && (g & (g - 1)) == 0; }

dq_status check_i8(const int8_t* x, const float* x_scales, const int32_t* x_sums, int64_t M,
                   int64_t max_m, const uint32_t* packed, const float* scales,
                   const int32_t* zeros, int64_t N, int64_t K, int32_t bits, const void* y,
                   int32_t y_dtype)
{
    if (!x || !x_scales || !x_sums || !packed || !scales || !y) return DQ_ERR_NULL;
    if (bits < DQ_MIN_BITS || bits > DQ_MAX_BITS_I8) return DQ_ERR_BITS;
    if (N < 1 || N > 0x7fffffffLL || K < 1 || K > DQ_MAX_K_I8 || M < 1 || M > max_m)
        return DQ_ERR_SHAPE;
    if (y_dtype != DQ_F32 && y_dtype != DQ_BF16) return DQ_ERR_DTYPE;
    if (!aligned(x, 16) || !aligned(packed, 16) || !aligned(x_scales, 4) || !aligned(x_sums, 4) ||
        !aligned(scales, 4) || !aligned(zeros, 4) || !aligned(y, y_dtype == DQ_BF16 ? 2 : 4))
        return DQ_ERR_ALIGN;
    return DQ_OK;
}

dq_status cache4_geometry(const dq_cache4* cache, dq::Cache4* c)
{
    const int32_t D = cache->head_dim, P = cache->page_size, g = cache->group;
    if ((D != 64 && D != 128 && D != 256) || P < 16 || P > 256 || (P & (P - 1)) != 0 ||
        (g != 32 && g != 64 && g != 128) || g > D || cache->kv_heads < 1 ||
        cache->kv_heads > DQ_CACHE4_MAX_HEADS || cache->pages < 1 || cache->pages > 0x7fffffffLL)
        return DQ_ERR_SHAPE;
    *c = dq::Cache4{cache->k_codes, cache->v_codes,  cache->k_scales, cache->v_scales,
                    cache->pages,   cache->kv_heads, D,               __builtin_ctz(P),
                    g};
    return DQ_OK;
}

dq_status check_cache4(const dq_cache4* cache, const dq_cache4_batch* batch, int64_t tokens,
                       dq::Cache4* c, dq::Cache4Batch* bt)
{
    if (!cache || !batch || !cache->k_codes || !cache->v_codes || !cache->k_scales ||
        !cache->v_scales || !batch->starts || !batch->lens || !batch->table)
        return DQ_ERR_NULL;
    const dq_status st = cache4_geometry(cache, c);
    if (st != DQ_OK) return st;
    if (batch->count < 1 || batch->count > DQ_CACHE4_MAX_COUNT || batch->table_width < 1 ||
        batch->table_width > (1LL << 24) || tokens < 1 || tokens > 0x7fffffffLL)
        return DQ_ERR_SHAPE;
    if (!aligned(cache->k_codes, 16) || !aligned(cache->v_codes, 16) ||
        !aligned(cache->k_scales, 16) || !aligned(cache->v_scales, 16) ||
        !aligned(batch->starts, 4) || !aligned(batch->lens, 4) || !aligned(batch->table, 4))
        return DQ_ERR_ALIGN;
    *bt = dq::Cache4Batch{batch->starts, batch->lens, batch->table, batch->table_width, batch->count};
    return DQ_OK;
}

bool valid_stride(int64_t stride, int64_t row)
{
    return stride >= row && stride <= (1LL << 32) && stride % 8 == 0;
}

bool valid_heads(int32_t q_heads, int32_t kv_heads)
{
    return q_heads >= 1 && q_heads <= DQ_CACHE4_MAX_HEADS && q_heads % kv_heads == 0;
}

}  // namespace

int32_t dq::record_hip_error(hipError_t e) { return hip_status(e); }

extern "C" {

size_t dq_packed_row_bytes(int64_t K, int32_t bits)
{
    if (bits < DQ_MIN_BITS || bits > DQ_MAX_BITS || K < 1 || K > DQ_MAX_K) return 0;
    return (size_t)dq::packed_row_words(K, bits) * 4;
}

dq_status dq_quantize_pack(const void* w, int32_t w_dtype, int64_t N, int64_t K, int32_t bits,
                           uint32_t* packed, float* scales, uint32_t* nonfinite_rows,
                           void* stream)
{
    if (!w || !packed || !scales) return DQ_ERR_NULL;
    dq_status st = check_common(N, K, bits);
    if (st != DQ_OK) return st;
    if (w_dtype != DQ_F32 && w_dtype != DQ_BF16) return DQ_ERR_DTYPE;
    if (!aligned(w, 16) || !aligned(packed, 16) || !aligned(scales, 4) ||
        !aligned(nonfinite_rows, 4))
        return DQ_ERR_ALIGN;
    return hip_status(dq::launch_quantize_pack(w, w_dtype == DQ_BF16, N, K, bits, packed, scales,
                                               nonfinite_rows, static_cast<hipStream_t>(stream)));
}

dq_status dq_quantize_pack_sumsq(const void* w, int32_t w_dtype, int64_t N, int64_t K,
                                 int32_t bits, uint32_t* packed, float* scales,
                                 double* row_sumsq, double* matrix_sumsq, void* stream)
{
    if (!w || !packed || !scales || !row_sumsq) return DQ_ERR_NULL;
    dq_status st = check_common(N, K, bits);
    if (st != DQ_OK) return st;
    if (w_dtype != DQ_F32 && w_dtype != DQ_BF16) return DQ_ERR_DTYPE;
    if (!aligned(w, 16) || !aligned(packed, 16) || !aligned(scales, 4) || !aligned(row_sumsq, 8) ||
        !aligned(matrix_sumsq, 8))
        return DQ_ERR_ALIGN;
    return hip_status(dq::launch_quantize_pack_sumsq(w, w_dtype == DQ_BF16, N, K, bits, packed,
                                                     scales, row_sumsq, matrix_sumsq,
                                                     static_cast<hipStream_t>(stream)));
}

dq_status dq_row_sumsq(const void* w, int32_t w_dtype, int64_t N, int64_t K, double* row_sumsq,
                       double* matrix_sumsq, void* stream)
{
    if (!w || !row_sumsq) return DQ_ERR_NULL;
    if (N < 1 || N > 0x7fffffffLL || K < 1 || K > DQ_MAX_K) return DQ_ERR_SHAPE;
    if (w_dtype != DQ_F32 && w_dtype != DQ_BF16) return DQ_ERR_DTYPE;
    if (!aligned(w, 16) || !aligned(row_sumsq, 8) || !aligned(matrix_sumsq, 8))
        return DQ_ERR_ALIGN;
    return hip_status(dq::launch_row_sumsq(w, w_dtype == DQ_BF16, N, K, row_sumsq, matrix_sumsq,
                                           static_cast<hipStream_t>(stream)));
}

dq_status dq_unpack(const uint32_t* packed, const float* scales, int64_t N, int64_t K,
                    int32_t bits, int32_t* q_out, float* w_out, void* stream)
{
    if (!packed || (!q_out && !w_out) || (w_out && !scales)) return DQ_ERR_NULL;
    dq_status st = check_common(N, K, bits);
    if (st != DQ_OK) return st;
    if (!aligned(packed, 16) || !aligned(scales, 4) || !aligned(q_out, 4) || !aligned(w_out, 4))
        return DQ_ERR_ALIGN;
    return hip_status(dq::launch_unpack(packed, scales, nullptr, 0, N, K, bits, q_out, w_out,
                                        static_cast<hipStream_t>(stream)));
}

dq_status dq_quantize_pack_asym(const void* w, int32_t w_dtype, int64_t N, int64_t K, int32_t bits,
                                uint32_t* packed, float* scales, int32_t* zeros, void* stream)
{
    if (!w || !packed || !scales || !zeros) return DQ_ERR_NULL;
    dq_status st = check_common(N, K, bits);
    if (st != DQ_OK) return st;
    if (w_dtype != DQ_F32 && w_dtype != DQ_BF16) return DQ_ERR_DTYPE;
    if (!aligned(w, 16) || !aligned(packed, 16) || !aligned(scales, 4) || !aligned(zeros, 4))
        return DQ_ERR_ALIGN;
    return hip_status(dq::launch_quantize_pack_asym(w, w_dtype == DQ_BF16, N, K, bits, packed,
                                                    scales, zeros,
                                                    static_cast<hipStream_t>(stream)));
}

dq_status dq_unpack_asym(const uint32_t* packed, const float* scales, const int32_t* zeros,
                         int64_t N, int64_t K, int32_t bits, int32_t* q_out, float* w_out,
                         void* stream)
{
    if (!packed || !zeros || (!q_out && !w_out) || (w_out && !scales)) return DQ_ERR_NULL;
    dq_status st = check_common(N, K, bits);
    if (st != DQ_OK) return st;
    if (!aligned(packed, 16) || !aligned(scales, 4) || !aligned(zeros, 4) || !aligned(q_out, 4) ||
        !aligned(w_out, 4))
        return DQ_ERR_ALIGN;
    return hip_status(dq::launch_unpack(packed, scales, zeros, 0, N, K, bits, q_out, w_out,
                                        static_cast<hipStream_t>(stream)));
}

dq_status dq_quantize_pack_group(const void* w, int32_t w_dtype, int64_t N, int64_t K,
                                 int32_t bits, int64_t group, uint32_t* packed, float* scales,
                                 void* stream)
{
    if (!w || !packed || !scales) return DQ_ERR_NULL;
    dq_status st = check_common(N, K, bits);
    if (st != DQ_OK) return st;
    if (!valid_group(group)) return DQ_ERR_SHAPE;
    if (w_dtype != DQ_F32 && w_dtype != DQ_BF16) return DQ_ERR_DTYPE;
    if (!aligned(w, 16) || !aligned(packed, 16) || !aligned(scales, 4)) return DQ_ERR_ALIGN;
    return hip_status(dq::launch_quantize_pack_group(w, w_dtype == DQ_BF16, N, K, bits, group,
                                                     packed, scales,
                                                     static_cast<hipStream_t>(stream)));
}

dq_status dq_unpack_group(const uint32_t* packed, const float* scales, int64_t N, int64_t K,
                          int32_t bits, int64_t group, int32_t* q_out, float* w_out, void* stream)
{
    if (!packed || (!q_out && !w_out) || (w_out && !scales)) return DQ_ERR_NULL;
    dq_status st = check_common(N, K, bits);
    if (st != DQ_OK) return st;
    if (!valid_group(group)) return DQ_ERR_SHAPE;
    if (!aligned(packed, 16) || !aligned(scales, 4) || !aligned(q_out, 4) || !aligned(w_out, 4))
        return DQ_ERR_ALIGN;
    return hip_status(dq::launch_unpack(packed, scales, nullptr, group, N, K, bits, q_out, w_out,
                                        static_cast<hipStream_t>(stream)));
}

dq_status dq_gemv_group(const uint16_t* x, int64_t M, const uint32_t* packed, const float* scales,
                        int64_t N, int64_t K, int32_t bits, int64_t group, float* y, void* stream)
{
    if (!x || !packed || !scales || !y) return DQ_ERR_NULL;
    dq_status st = check_common(N, K, bits);
    if (st != DQ_OK) return st;
    if (M < 1 || M > DQ_GEMV_MAX_M || !valid_group(group)) return DQ_ERR_SHAPE;
    if (!aligned(x, 16) || !aligned(packed, 16) || !aligned(scales, 4) || !aligned(y, 4))
        return DQ_ERR_ALIGN;
    return hip_status(dq::launch_gemv_group(x, M, packed, scales, N, K, bits, group, y,
                                            static_cast<hipStream_t>(stream)));
}

dq_status dq_gemm_group(const uint16_t* x, int64_t M, const uint32_t* packed, const float* scales,
                        int64_t N, int64_t K, int32_t bits, int64_t group, float* y, void* stream)
{
    if (!x || !packed || !scales || !y) return DQ_ERR_NULL;
    dq_status st = check_common(N, K, bits);
    if (st != DQ_OK) return st;
    if (M < 1 || M > 0x7fffffffLL || !valid_group(group)) return DQ_ERR_SHAPE;
    if (!aligned(x, 16) || !aligned(packed, 16) || !aligned(scales, 4) || !aligned(y, 4))
        return DQ_ERR_ALIGN;
    return hip_status(dq::launch_gemm_group(x, M, packed, scales, N, K, bits, group, y,
                                            static_cast<hipStream_t>(stream)));
}

dq_status dq_gemv(const uint16_t* x, int64_t M, const uint32_t* packed, const float* scales,
                  int64_t N, int64_t K, int32_t bits, float* y, void* stream)
{
    if (!x || !packed || !scales || !y) return DQ_ERR_NULL;
    dq_status st = check_common(N, K, bits);
    if (st != DQ_OK) return st;
    if (M < 1 || M > DQ_GEMV_MAX_M) return DQ_ERR_SHAPE;
    if (!aligned(x, 16) || !aligned(packed, 16) || !aligned(scales, 4) || !aligned(y, 4))
        return DQ_ERR_ALIGN;
    return hip_status(dq::launch_gemv(x, M, packed, scales, N, K, bits, y, nullptr,
                                      static_cast<hipStream_t>(stream)));
}

dq_status dq_gemv_batched(const dq_gemv_item* items, int32_t count, int64_t M, void* stream)
{
    if (!items) return DQ_ERR_NULL;
    if (count < 1 || count > DQ_GEMV_BATCH_MAX || M < 1 || M > DQ_GEMV_MAX_M) return DQ_ERR_SHAPE;
    static_assert(DQ_GEMV_BATCH_MAX == dq::kGemvBatchMax, "batch size");
    dq::GemvItem g[DQ_GEMV_BATCH_MAX];
    for (int32_t i = 0; i < count; ++i) {  // every item is checked before anything is enqueued
        const dq_gemv_item& it = items[i];
        if (!it.x || !it.packed || !it.scales || !it.y) return DQ_ERR_NULL;
        const dq_status st = check_common(it.N, it.K, it.bits);
        if (st != DQ_OK) return st;
        if (it.group != 0 && (!valid_group(it.group) || it.zeros)) return DQ_ERR_SHAPE;
        if (!aligned(it.x, 16) || !aligned(it.packed, 16) || !aligned(it.scales, 4) ||
            !aligned(it.y, 4) || !aligned(it.zeros, 4))
            return DQ_ERR_ALIGN;
        g[i] = dq::GemvItem{it.x, it.packed, it.scales, it.y, it.N, it.K, it.bits, it.group, it.zeros};
    }
    return hip_status(dq::launch_gemv_batched(g, count, M, static_cast<hipStream_t>(stream)));
}

dq_status dq_gemv_asym(const uint16_t* x, int64_t M, const uint32_t* packed, const float* scales,
                       const int32_t* zeros, int64_t N, int64_t K, int32_t bits, float* y,
                       void* stream)
{
    if (!x || !packed || !scales || !zeros || !y) return DQ_ERR_NULL;
    dq_status st = check_common(N, K, bits);
    if (st != DQ_OK) return st;
    if (M < 1 || M > DQ_GEMV_MAX_M) return DQ_ERR_SHAPE;
    if (!aligned(x, 16) || !aligned(packed, 16) || !aligned(scales, 4) || !aligned(y, 4) ||
        !aligned(zeros, 4))
        return DQ_ERR_ALIGN;
    return hip_status(dq::launch_gemv(x, M, packed, scales, N, K, bits, y, zeros,
                                      static_cast<hipStream_t>(stream)));
}

dq_status dq_gemm(const uint16_t* x, int64_t M, const uint32_t* packed, const float* scales,
                  int64_t N, int64_t K, int32_t bits, float* y, void* stream)
{
    if (!x || !packed || !scales || !y) return DQ_ERR_NULL;
    dq_status st = check_common(N, K, bits);
    if (st != DQ_OK) return st;
    if (M < 1 || M > 0x7fffffffLL) return DQ_ERR_SHAPE;
    if (!aligned(x, 16) || !aligned(packed, 16) || !aligned(scales, 4) || !aligned(y, 4))
        return DQ_ERR_ALIGN;
    return hip_status(dq::launch_gemm(x, M, packed, scales, N, K, bits, y, nullptr,
                                      static_cast<hipStream_t>(stream)));
}

dq_status dq_gemm_asym(const uint16_t* x, int64_t M, const uint32_t* packed, const float* scales,
                       const int32_t* zeros, int64_t N, int64_t K, int32_t bits, float* y,
                       void* stream)
{
    if (!x || !packed || !scales || !zeros || !y) return DQ_ERR_NULL;
    dq_status st = check_common(N, K, bits);
    if (st != DQ_OK) return st;
    if (M < 1 || M > 0x7fffffffLL) return DQ_ERR_SHAPE;
    if (!aligned(x, 16) || !aligned(packed, 16) || !aligned(scales, 4) || !aligned(y, 4) ||
        !aligned(zeros, 4))
        return DQ_ERR_ALIGN;
    return hip_status(dq::launch_gemm(x, M, packed, scales, N, K, bits, y, zeros,
                                      static_cast<hipStream_t>(stream)));
}

dq_status dq_file_load(const dq_file* f, int64_t i, void* data, float* scales, void* stream)
{
    if (!f || !data) return DQ_ERR_NULL;
    dq_file_matrix m;
    const dq_status st = dq_file_matrix_info(f, i, &m);
    if (st != DQ_OK) return st;
    if (m.scales && !scales) return DQ_ERR_NULL;
    if (!aligned(data, 16) || !aligned(scales, 4)) return DQ_ERR_ALIGN;
    // region sizes follow from the entry's shape, which dq_file_open checked
    // against the file's extent
    const uint64_t db = m.bits == DQ_TOP_BITS
                            ? (uint64_t)m.N * (uint64_t)m.K * 2
                            : (uint64_t)m.N * (uint64_t)dq::packed_row_words(m.K, m.bits) * 4;
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t err = hipMemcpyAsync(data, m.data, db, hipMemcpyHostToDevice, s);
    if (err == hipSuccess && m.scales)
        err = hipMemcpyAsync(scales, m.scales, (uint64_t)m.N * 4, hipMemcpyHostToDevice, s);
    return hip_status(err);
}

size_t dq_token_row_bytes(int64_t K)
{
    return K < 1 || K > DQ_MAX_K_I8 ? 0 : (size_t)dq::token_row_bytes(K);
}

dq_status dq_quantize_tokens(const void* x, int32_t x_dtype, int64_t M, int64_t K, int8_t* codes,
                             float* scales, int32_t* sums, void* stream)
{
    if (!x || !codes || !scales || !sums) return DQ_ERR_NULL;
    if (M < 1 || M > 0x7fffffffLL || K < 1 || K > DQ_MAX_K_I8) return DQ_ERR_SHAPE;
    if (x_dtype != DQ_F32 && x_dtype != DQ_BF16) return DQ_ERR_DTYPE;
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(sums, 4))
        return DQ_ERR_ALIGN;
    return hip_status(dq::launch_quantize_tokens(x, x_dtype == DQ_BF16, M, K, codes, scales, sums,
                                                 static_cast<hipStream_t>(stream)));
}

dq_status dq_gemv_i8(const int8_t* x, const float* x_scales, const int32_t* x_sums, int64_t M,
                     const uint32_t* packed, const float* scales, const int32_t* zeros, int64_t N,
                     int64_t K, int32_t bits, void* y, int32_t y_dtype, void* stream)
{
    const dq_status st = check_i8(x, x_scales, x_sums, M, DQ_GEMV_MAX_M, packed, scales, zeros, N,
                                  K, bits, y, y_dtype);
    if (st != DQ_OK) return st;
    return hip_status(dq::launch_gemm_i8(x, x_scales, x_sums, M, packed, scales, zeros, N, K, bits,
                                         y, y_dtype == DQ_BF16, static_cast<hipStream_t>(stream)));
}

dq_status dq_gemm_i8(const int8_t* x, const float* x_scales, const int32_t* x_sums, int64_t M,
                     const uint32_t* packed, const float* scales, const int32_t* zeros, int64_t N,
                     int64_t K, int32_t bits, void* y, int32_t y_dtype, void* stream)
{
    const dq_status st = check_i8(x, x_scales, x_sums, M, 0x7fffffffLL, packed, scales, zeros, N,
                                  K, bits, y, y_dtype);
    if (st != DQ_OK) return st;
    return hip_status(dq::launch_gemm_i8(x, x_scales, x_sums, M, packed, scales, zeros, N, K, bits,
                                         y, y_dtype == DQ_BF16, static_cast<hipStream_t>(stream)));
}

dq_status dq_cache4_append(const dq_cache4* cache, const dq_cache4_batch* batch, const void* k,
                           const void* v, int32_t dtype, int64_t tokens, int64_t k_stride,
                           int64_t v_stride, void* stream)
{
    if (!k || !v) return DQ_ERR_NULL;
    dq::Cache4 c;
    dq::Cache4Batch bt;
    const dq_status st = check_cache4(cache, batch, tokens, &c, &bt);
    if (st != DQ_OK) return st;
    const int64_t row = (int64_t)c.heads * c.dim;
    if (!valid_stride(k_stride, row) || !valid_stride(v_stride, row)) return DQ_ERR_SHAPE;
    if (dtype != DQ_F32 && dtype != DQ_BF16) return DQ_ERR_DTYPE;
    if (!aligned(k, 16) || !aligned(v, 16)) return DQ_ERR_ALIGN;
    return hip_status(dq::launch_cache4_append(c, bt, k, v, dtype == DQ_BF16, tokens, k_stride,
                                               v_stride, static_cast<hipStream_t>(stream)));
}

dq_status dq_cache4_read(const dq_cache4* cache, const dq_cache4_batch* batch, void* k, void* v,
                         int32_t dtype, int64_t tokens, void* stream)
{
    if (!k || !v) return DQ_ERR_NULL;
    dq::Cache4 c;
    dq::Cache4Batch bt;
    const dq_status st = check_cache4(cache, batch, tokens, &c, &bt);
    if (st != DQ_OK) return st;
    if (dtype != DQ_F32 && dtype != DQ_BF16) return DQ_ERR_DTYPE;
    if (!aligned(k, 16) || !aligned(v, 16)) return DQ_ERR_ALIGN;
    return hip_status(dq::launch_cache4_read(c, bt, k, v, dtype == DQ_BF16, tokens,
                                             static_cast<hipStream_t>(stream)));
}

size_t dq_cache4_attention_workspace(const dq_cache4* cache, int64_t count, int64_t tokens,
                                     int32_t q_heads, int64_t max_q, int64_t max_len)
{
    dq::Cache4 c;
    if (!cache || cache4_geometry(cache, &c) != DQ_OK || count < 1 || count > DQ_CACHE4_MAX_COUNT ||
        tokens < 1 || tokens > 0x7fffffffLL || !valid_heads(q_heads, c.heads) || max_q < 1 || max_len < 1)
        return 0;
    return dq::cache4_attention_workspace(c, count, tokens, q_heads, max_q, max_len);
}

dq_status dq_cache4_attention(const dq_cache4* cache, const dq_cache4_batch* batch,
                              const uint16_t* q, int64_t tokens, int64_t q_stride, int32_t q_heads,
                              float scale, int64_t max_q, int64_t max_len, uint16_t* out,
                              void* workspace, size_t workspace_bytes, void* stream)
{
    if (!q || !out) return DQ_ERR_NULL;
    dq::Cache4 c;
    dq::Cache4Batch bt;
    const dq_status st = check_cache4(cache, batch, tokens, &c, &bt);
    if (st != DQ_OK) return st;
    if (!valid_heads(q_heads, c.heads) || !valid_stride(q_stride, (int64_t)q_heads * c.dim) ||
        max_q < 1 || max_len < 1)
        return DQ_ERR_SHAPE;
    if (!std::isfinite(scale * 1.44269504f)) return DQ_ERR_VALUE;  // exp2's argument is scaled
    const size_t need = dq::cache4_attention_workspace(c, bt.count, tokens, q_heads, max_q, max_len);
    if (need && !workspace) return DQ_ERR_NULL;
    if (need > workspace_bytes) return DQ_ERR_SHAPE;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16)) return DQ_ERR_ALIGN;
    return hip_status(dq::launch_cache4_attention(c, bt, q, tokens, q_stride, q_heads, scale, max_q,
                                                  max_len, out, workspace,
                                                  static_cast<hipStream_t>(stream)));
}

dq_status dq_stream_read(const void* buf, int64_t bytes, uint32_t* partial, int64_t nparts,
                         void* stream)
{
    if (!buf || !partial) return DQ_ERR_NULL;
    if (bytes < 16 || bytes % 16 != 0 || nparts < 1 || nparts > DQ_STREAM_MAX_PARTS)
        return DQ_ERR_SHAPE;
    if (!aligned(buf, 16) || !aligned(partial, 4)) return DQ_ERR_ALIGN;
    return hip_status(
        dq::launch_stream_read(buf, bytes, partial, nparts, static_cast<hipStream_t>(stream)));
}

const char* dq_status_string(dq_status status)
{
    switch (status) {
    case DQ_OK: return "ok";
    case DQ_ERR_NULL: return "a required pointer is NULL";
    case DQ_ERR_BITS: return "bits must be in [2, 15] (integer products: [2, 8]; allocation levels: increasing, in [2, 16])";
    case DQ_ERR_SHAPE: return "N, K, M, or a cache's sizes, heads, strides or workspace out of range";
    case DQ_ERR_ALIGN:
        return "pointer not aligned (W, packed, x, token codes, cache, q, k, v: 16 bytes; fp64 sums: 8; others: their elements)";
    case DQ_ERR_DTYPE: return "a dtype must be DQ_F32 or DQ_BF16";
    case DQ_ERR_HIP: return "HIP launch or runtime error";
    case DQ_ERR_BUDGET: return "bit budget below every matrix at its lowest level";
    case DQ_ERR_VALUE:
        return "sensitivity, trace or sum not finite and >= 0, scale not finite, parameter count out of range, or "
               "a name without its terminating NUL";
    case DQ_ERR_IO: return "file could not be opened, written, sized or mapped";
    case DQ_ERR_FORMAT: return "file is not a packed-weight file of this version, or is corrupt";
    default: return "unknown status";
    }
}

const char* dq_last_error(void) { return g_last_error; }

}  // extern "C"
