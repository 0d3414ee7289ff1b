// Filling and reading the paged 4-bit key/value cache (geometry: cache4.hpp).
// A head's vector is quantized as a row of the group-wise quantizer at b = 4
// ("量化" tutorial, aiknowledge.cn, exercise 1 of its exercises): per group of g
// dimensions s = fl32(max / 7) (1.0 replaces a zero max), q = clip(rint(fl32(
// v / s)), -8, 7), code u = q + 8; a group with a NaN or an infinity gets a NaN
// scale and q = 0.
//
// A thread owns 8 dimensions of one (token, kv head, keys or values) row, so a
// row is D/8 neighbouring threads of a wave and a group g/8 of them: the
// group's maximum is a butterfly over those lanes.
#include "cache4.hpp"
#include "common.hpp"
#include "launch_serving.hpp"
#include "quant_rule.hpp"

namespace dq {

namespace {

constexpr int kThreads = 256;

// The row that a thread works on: row = (token * heads + head) * 2 + (0 keys, 1 values).
struct RowAt {
    int64_t token;
    int head;
    bool value;
    int part;  // which 8 dimensions
};

__device__ __forceinline__ RowAt row_at(const Cache4& c, int64_t row, int part)
{
    const int64_t th = row >> 1;
    return RowAt{th / c.heads, (int)(th % c.heads), (row & 1) != 0, part};
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void cache4_append_kernel(
    Cache4 c, Cache4Batch bt, const void* __restrict__ k, const void* __restrict__ v,
    int64_t tokens, int64_t k_stride, int64_t v_stride)
{
    __shared__ uint8_t nib[kThreads * 8];
    const int parts = c.dim >> 3;  // threads of a row: 8, 16 or 32
    const int rows_here = kThreads / parts;
    const int local = threadIdx.x / parts;
    const RowAt at = row_at(c, (int64_t)blockIdx.x * rows_here + local, threadIdx.x % parts);
    int64_t slot = -1;
    bool live = at.token < tokens && cache4_slot(c, bt, at.token, tokens, &slot);
    live = live && slot >= 0;

    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.0f;
    if (live) {
        const int64_t off = at.token * (at.value ? v_stride : k_stride) + at.head * c.dim + at.part * 8;
        const void* src = at.value ? v : k;
        if (BF16) {
            const uint4 d = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(src) + off);
            const uint32_t u[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[2 * e] = __uint_as_float(u[e] << 16);
                x[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
            }
        } else {
            const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(src) + off);
            const float4 a = p[0], b = p[1];
            x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
            x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
        }
    }
    uint32_t amax = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t a = __float_as_uint(x[e]) & 0x7fffffffu;
        amax = a > amax ? a : amax;
    }
    for (int o = c.group >> 4; o > 0; o >>= 1) {
        const uint32_t t = (uint32_t)__shfl_xor((int)amax, o, kWave);
        amax = t > amax ? t : amax;
    }
    float s;
    bool zero = false;
    if (amax >= 0x7f800000u) {
        s = __uint_as_float(0x7fc00000u);
        zero = true;
    } else {
        const float a = __uint_as_float(amax);
        s = (a == 0.0f ? 1.0f : a) / 7.0f;
        if (a == 0.0f || s == 0.0f) {
            s = 1.0f / 7.0f;
            zero = true;
        }
    }
    const float r = 1.0f / s;
    const float margin = quotient_margin(8.0f);
    uint32_t word = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float q = fminf(fmaxf(rounded_quotient(x[e], s, r, margin), -8.0f), 7.0f);
        const uint32_t u = zero ? 8u : (uint32_t)((int32_t)q + 8);
        nib[threadIdx.x * 8 + e] = (uint8_t)u;
        word |= u << (4 * e);
    }
    __syncthreads();  // a row's threads are inside one wave, but rows share no order otherwise
    if (!live) return;
    const int64_t page = slot >> c.page_shift;
    const int64_t off = slot & ((1LL << c.page_shift) - 1);
    const int64_t block = page * c.heads + at.head;  // (page, head)
    const int64_t row = ((block << c.page_shift) + off) * parts;
    if (!at.value) {
        // dimensions 8 part .. = 32 i + 8 r: word r (D/32) + i
        c.k_codes[row + (at.part & 3) * (c.dim >> 5) + (at.part >> 2)] = word;
    } else {
        // word w of the row holds codes 8 w .. 8 w + 7; code n is dimension 16 j + c, n = c (D/16) + j
        const int per = c.dim >> 4;
        const uint8_t* src = nib + local * c.dim;
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int n = at.part * 8 + e;
            w |= (uint32_t)src[16 * (n % per) + n / per] << (4 * e);
        }
        c.v_codes[row + at.part] = w;
    }
    const int gp = c.group >> 3;  // threads of a group
    if (at.part % gp == 0) {
        const int groups = c.dim / c.group;
        float* dst = at.value ? c.v_scales : c.k_scales;
        dst[((block * groups + at.part / gp) << c.page_shift) + off] = s;
    }
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void cache4_read_kernel(Cache4 c, Cache4Batch bt,
                                                               void* __restrict__ k,
                                                               void* __restrict__ v, int64_t tokens)
{
    const int parts = c.dim >> 3;
    const int rows_here = kThreads / parts;
    const RowAt at = row_at(c, (int64_t)blockIdx.x * rows_here + threadIdx.x / parts,
                            threadIdx.x % parts);
    int64_t slot = -1;
    if (at.token >= tokens || !cache4_slot(c, bt, at.token, tokens, &slot)) return;
    float x[8];
    if (slot < 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(0x7fc00000u);
    } else {
        const int64_t page = slot >> c.page_shift;
        const int64_t off = slot & ((1LL << c.page_shift) - 1);
        const int64_t block = page * c.heads + at.head;
        const int64_t row = ((block << c.page_shift) + off) * parts;
        const int groups = c.dim / c.group;
        const float* sc = at.value ? c.v_scales : c.k_scales;
        const float s = sc[((block * groups + at.part * 8 / c.group) << c.page_shift) + off];
        if (!at.value) {
            const uint32_t w = c.k_codes[row + (at.part & 3) * (c.dim >> 5) + (at.part >> 2)];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = (float)((int32_t)((w >> (4 * e)) & 15u) - 8) * s;
        } else {
            const int per = c.dim >> 4;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int d = at.part * 8 + e;
                const int n = (d & 15) * per + (d >> 4);
                x[e] = (float)((int32_t)((c.v_codes[row + (n >> 3)] >> (4 * (n & 7))) & 15u) - 8) * s;
            }
        }
    }
    const int64_t o = (at.token * c.heads + at.head) * c.dim + at.part * 8;
    void* dst = at.value ? v : k;
    if (BF16) {
        uint32_t u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            u[e] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * e]) |
                   ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * e + 1]) << 16);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(dst) + o) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(dst) + o);
        p[0] = make_float4(x[0], x[1], x[2], x[3]);
        p[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
}

// One workgroup per kThreads / (D/8) rows of (token, head, keys | values).
bool row_grid(const Cache4& c, int64_t tokens, unsigned* grid)
{
    const int64_t rows = tokens * c.heads * 2;
    const int64_t blocks = ceil_div(rows, kThreads / (c.dim >> 3));
    if (blocks > 0x7fffffffLL) return false;
    *grid = (unsigned)blocks;
    return true;
}

}  // namespace

hipError_t launch_cache4_append(const Cache4& c, const Cache4Batch& bt, const void* k,
                                const void* v, bool bf16, int64_t tokens, int64_t k_stride,
                                int64_t v_stride, hipStream_t stream)
{
    unsigned grid;
    if (!row_grid(c, tokens, &grid)) return hipErrorInvalidConfiguration;
    if (bf16)
        cache4_append_kernel<true><<<grid, kThreads, 0, stream>>>(c, bt, k, v, tokens, k_stride, v_stride);
    else
        cache4_append_kernel<false><<<grid, kThreads, 0, stream>>>(c, bt, k, v, tokens, k_stride, v_stride);
    return hipGetLastError();
}

hipError_t launch_cache4_read(const Cache4& c, const Cache4Batch& bt, void* k, void* v, bool bf16,
                              int64_t tokens, hipStream_t stream)
{
    unsigned grid;
    if (!row_grid(c, tokens, &grid)) return hipErrorInvalidConfiguration;
    if (bf16)
        cache4_read_kernel<true><<<grid, kThreads, 0, stream>>>(c, bt, k, v, tokens);
    else
        cache4_read_kernel<false><<<grid, kThreads, 0, stream>>>(c, bt, k, v, tokens);
    return hipGetLastError();
}

}  // namespace dq
