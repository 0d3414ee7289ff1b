// Filling and reading the paged 4-bit key/value cache (geometry: cache4.hpp).
// A head's vector is quantized as a row of the group-wise quantizer at b = 4
// ("量化" tutorial, aiknowledge.cn, exercise 1 of its exercises): per group of g
// dimensions s = fl32(max / 7) (1.0 replaces a zero max), q = clip(rint(fl32(
// v / s)), -8, 7), code u = q + 8; a group with a NaN or an infinity gets a NaN
// scale and q = 0.
//
// Both kernels are bound by memory.  A workgroup has kTokens consecutive tokens, so
// where a token lives is worked out once, with scalars, while its elements are on
// their way; a thread has 8 dimensions of a (kv head, keys or values) row, D/8
// neighbouring threads of a wave a row, g/8 of them a group, whose maximum is a
// butterfly over those lanes.  6207 tokens of 8 heads of 128 in bf16 (a token
// each for a workgroup of as many threads, its place found by every thread, took
// 27 us to append and 19 us to read).
#include "cache4.hpp"
#include "common.hpp"
#include "launch_serving.hpp"
#include "quant_rule.hpp"

namespace dq {

namespace {

constexpr int kThreads = 256;

// The place of each of a workgroup's tokens from t0 on: -2 for a token of no
// sequence (or past the call's), -1 for one that the cache does not hold.
template <int kTokens>
__device__ __forceinline__ void find_slots(const Cache4& c, const Cache4Batch& bt, int64_t t0,
                                           int64_t tokens, int64_t (&slot)[kTokens])
{
    // token i of them by the lanes whose number is i modulo kTokens
    const int64_t t = t0 + (kTokens > 1 ? threadIdx.x % kTokens : 0);
    const int64_t b = cache4_sequence(bt, t);
    int64_t first, n, at = -2;
    cache4_rows(bt, b, tokens, first, n);
    if (t >= first && t < first + n)
        at = cache4_slot(c, bt, b, (int64_t)bt.lens[b] - n + (t - first));
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)at, i);
        const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(at >> 32), i);
        slot[i] = (int64_t)((uint64_t)hi << 32 | lo);
    }
}

// This thread's row (head, keys or values) and 8 dimensions; false past the last.
struct Part {
    int head;
    bool value;
    int part;
};
template <int D>
__device__ __forceinline__ bool part_of(const Cache4& c, Part* p)
{
    constexpr unsigned kParts = D / 8;
    const unsigned row = (blockIdx.y * blockDim.x + threadIdx.x) / kParts;
    p->part = threadIdx.x % kParts;
    p->value = row & 1;
    p->head = (int)(row >> 1);
    return p->head < c.heads;
}

template <int D, bool BF16, int kTokens>
__global__ __launch_bounds__(kThreads) void cache4_append_kernel(
    Cache4 c, Cache4Batch bt, const void* __restrict__ k, const void* __restrict__ v,
    int64_t tokens, int64_t k_stride, int64_t v_stride)
{
    constexpr int kParts = D / 8;
    constexpr int kPer = D / 16;  // value codes of a c (cache4.hpp)
    __shared__ __attribute__((aligned(16))) uint32_t turn[kThreads];
    const int64_t t0 = (int64_t)blockIdx.x * kTokens;
    Part at;
    const bool in = part_of<D>(c, &at);

    uint4 raw[kTokens][BF16 ? 1 : 2];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        raw[i][0] = make_uint4(0, 0, 0, 0);
        if constexpr (!BF16) raw[i][1] = make_uint4(0, 0, 0, 0);
        if (in && t0 + i < tokens) {
            const int64_t off = (t0 + i) * (at.value ? v_stride : k_stride) + at.head * D + at.part * 8;
            const uint4* src = reinterpret_cast<const uint4*>(
                static_cast<const char*>(at.value ? v : k) + off * (BF16 ? 2 : 4));
            raw[i][0] = src[0];
            if constexpr (!BF16) raw[i][1] = src[1];
        }
    }
    int64_t slot[kTokens];
    find_slots<kTokens>(c, bt, t0, tokens, slot);

    const float margin = quotient_margin(8.0f);
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        float x[8];
        const uint32_t u4[4] = {raw[i][0].x, raw[i][0].y, raw[i][0].z, raw[i][0].w};
        if constexpr (BF16) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[2 * e] = __uint_as_float(u4[e] << 16);
                x[2 * e + 1] = __uint_as_float(u4[e] & 0xffff0000u);
            }
        } else {
            const uint32_t w4[4] = {raw[i][1].x, raw[i][1].y, raw[i][1].z, raw[i][1].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[e] = __uint_as_float(u4[e]);
                x[4 + e] = __uint_as_float(w4[e]);
            }
        }
        uint32_t amax = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = max(amax, __float_as_uint(x[e]) & 0x7fffffffu);
        for (int o = c.group >> 4; o > 0; o >>= 1)
            amax = max(amax, (uint32_t)__shfl_xor((int)amax, o, kWave));
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
        float q[8];
        clipped_quotients(x, s, 1.0f / s, margin, 7.0f, q);
        // four codes at a time as the exact fp32 sum of 16^e (q + 8)
        float lo = 34952.0f, hi = 34952.0f;  // 0x8888
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            lo = fmaf(q[e], (float)(1 << (4 * e)), lo);
            hi = fmaf(q[4 + e], (float)(1 << (4 * e)), hi);
        }
        uint32_t word = (uint32_t)hi << 16 | (uint32_t)lo;
        if (zero) word = 0x88888888u;
        // values: dimension 8 part + e is 16 j + c with j = part / 2, c = 8 (part & 1)
        // + e; a row's words change hands through LDS, those of one half of the
        // c's next to each other
        // (a row is within a wave, whose LDS accesses are in order)
        const int row0 = threadIdx.x - at.part;
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        turn[row0 + (at.part & 1) * kPer + (at.part >> 1)] = word;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (!in || slot[i] < 0) continue;
        const int64_t page = slot[i] >> c.page_shift;
        const int64_t off = slot[i] & ((1LL << c.page_shift) - 1);
        const int64_t block = page * c.heads + at.head;  // (page, head)
        const int64_t row = ((block << c.page_shift) + off) * kParts;
        if (!at.value) {
            // dimensions 8 part .. = 32 i + 8 r: word r (D/32) + i
            c.k_codes[row + (at.part & 3) * (D / 32) + (at.part >> 2)] = word;
        } else {
            // word w holds the codes 8 w + n: dimension 16 j + c for 8 w + n = c (D/16) + j
            constexpr int kRun = kPer < 8 ? kPer : 8;  // codes of one c in the word
            const int c0 = at.part * 8 / kPer;
            const uint4* from = reinterpret_cast<const uint4*>(
                &turn[row0 + (c0 >> 3) * kPer + at.part * 8 % kPer]);
            uint32_t x8[kRun];
#pragma unroll
            for (int e = 0; e < kRun; e += 4) {
                const uint4 d = from[e / 4];
                x8[e] = d.x, x8[e + 1] = d.y, x8[e + 2] = d.z, x8[e + 3] = d.w;
            }
            uint32_t w = 0;
#pragma unroll
            for (int n = 0; n < 8; ++n)
                w |= ((x8[n % kRun] >> (4 * ((c0 + n / kRun) & 7))) & 15u) << (4 * n);
            c.v_codes[row + at.part] = w;
        }
        const int gp = c.group >> 3;  // threads of a group
        if ((at.part & (gp - 1)) == 0) {
            float* dst = at.value ? c.v_scales : c.k_scales;
            dst[((block * (D / c.group) + at.part / gp) << c.page_shift) + off] = s;
        }
    }
}

template <int D, bool BF16, int kTokens>
__global__ __launch_bounds__(kThreads) void cache4_read_kernel(Cache4 c, Cache4Batch bt,
                                                               void* __restrict__ k,
                                                               void* __restrict__ v, int64_t tokens)
{
    constexpr int kParts = D / 8;
    constexpr int kWords = D / 64 * 4;  // of the 8 c's of a thread's dimensions
    const int64_t t0 = (int64_t)blockIdx.x * kTokens;
    Part at;
    const bool in = part_of<D>(c, &at);
    int64_t slot[kTokens];
    find_slots<kTokens>(c, bt, t0, tokens, slot);
    if (!in) return;

    uint32_t w[kTokens][kWords];
    float s[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        if (slot[i] < 0) continue;
        const int64_t page = slot[i] >> c.page_shift;
        const int64_t off = slot[i] & ((1LL << c.page_shift) - 1);
        const int64_t block = page * c.heads + at.head;
        const int64_t row = ((block << c.page_shift) + off) * kParts;
        if (!at.value) {
            w[i][0] = c.k_codes[row + (at.part & 3) * (D / 32) + (at.part >> 2)];
        } else {
            const uint4* src = reinterpret_cast<const uint4*>(c.v_codes + row + (at.part & 1) * kWords);
#pragma unroll
            for (int e = 0; e < kWords; e += 4) {
                const uint4 x = src[e / 4];
                w[i][e] = x.x, w[i][e + 1] = x.y, w[i][e + 2] = x.z, w[i][e + 3] = x.w;
            }
        }
        const float* sc = at.value ? c.v_scales : c.k_scales;
        s[i] = sc[((block * (D / c.group) + at.part * 8 / c.group) << c.page_shift) + off];
    }
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        if (slot[i] == -2) continue;
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            uint32_t u;
            if (!at.value) {
                u = w[i][0] >> (4 * e);
            } else {
                // code j = part / 2 of the e-th c
                const int j = at.part >> 1;
                if constexpr (D == 64)
                    u = w[i][e / 2] >> (16 * (e & 1) + 4 * j);
                else if constexpr (D == 128)
                    u = w[i][e] >> (4 * j);
                else
                    u = (j & 8 ? w[i][2 * e + 1] : w[i][2 * e]) >> (4 * (j & 7));
            }
            x[e] = slot[i] < 0 ? __uint_as_float(0x7fc00000u) : (float)((int32_t)(u & 15u) - 8) * s[i];
        }
        const int64_t o = ((t0 + i) * c.heads + at.head) * D + at.part * 8;
        void* dst = at.value ? v : k;
        if constexpr (BF16) {
            uint32_t p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                p[e] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * e]) |
                       ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * e + 1]) << 16);
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(dst) + o) = make_uint4(p[0], p[1], p[2], p[3]);
        } else {
            float4* p = reinterpret_cast<float4*>(static_cast<float*>(dst) + o);
            p[0] = make_float4(x[0], x[1], x[2], x[3]);
            p[1] = make_float4(x[4], x[5], x[6], x[7]);
        }
    }
}

// kTokens tokens by all rows of a token; a token each while there are fewer than
// fill the CUs four deep.
template <int kTokens>
bool token_grid(const Cache4& c, int64_t tokens, dim3* grid, unsigned* threads)
{
    const int64_t all = (int64_t)c.heads * 2 * (c.dim / 8);
    *threads = all >= kThreads ? kThreads : (unsigned)ceil_div(all, kWave) * kWave;
    const int64_t x = ceil_div(tokens, kTokens);
    *grid = dim3((unsigned)x, (unsigned)ceil_div(all, *threads));
    return x <= 0x7fffffffLL;
}

template <int D, bool BF16>
hipError_t append_d(const Cache4& c, const Cache4Batch& bt, const void* k, const void* v,
                    int64_t tokens, int64_t k_stride, int64_t v_stride, hipStream_t stream)
{
    dim3 grid;
    unsigned threads;
    if (tokens >= 4096) {
        if (!token_grid<4>(c, tokens, &grid, &threads)) return hipErrorInvalidConfiguration;
        cache4_append_kernel<D, BF16, 4><<<grid, threads, 0, stream>>>(c, bt, k, v, tokens, k_stride, v_stride);
    } else {
        if (!token_grid<1>(c, tokens, &grid, &threads)) return hipErrorInvalidConfiguration;
        cache4_append_kernel<D, BF16, 1><<<grid, threads, 0, stream>>>(c, bt, k, v, tokens, k_stride, v_stride);
    }
    return hipGetLastError();
}

template <int D, bool BF16>
hipError_t read_d(const Cache4& c, const Cache4Batch& bt, void* k, void* v, int64_t tokens,
                  hipStream_t stream)
{
    dim3 grid;
    unsigned threads;
    if (tokens >= 4096) {
        if (!token_grid<4>(c, tokens, &grid, &threads)) return hipErrorInvalidConfiguration;
        cache4_read_kernel<D, BF16, 4><<<grid, threads, 0, stream>>>(c, bt, k, v, tokens);
    } else {
        if (!token_grid<1>(c, tokens, &grid, &threads)) return hipErrorInvalidConfiguration;
        cache4_read_kernel<D, BF16, 1><<<grid, threads, 0, stream>>>(c, bt, k, v, tokens);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_cache4_append(const Cache4& c, const Cache4Batch& bt, const void* k,
                                const void* v, bool bf16, int64_t tokens, int64_t k_stride,
                                int64_t v_stride, hipStream_t stream)
{
#define CALL(D) \
    (bf16 ? append_d<D, true>(c, bt, k, v, tokens, k_stride, v_stride, stream) \
          : append_d<D, false>(c, bt, k, v, tokens, k_stride, v_stride, stream))
    return c.dim == 64 ? CALL(64) : (c.dim == 128 ? CALL(128) : CALL(256));
#undef CALL
}

hipError_t launch_cache4_read(const Cache4& c, const Cache4Batch& bt, void* k, void* v, bool bf16,
                              int64_t tokens, hipStream_t stream)
{
#define CALL(D) \
    (bf16 ? read_d<D, true>(c, bt, k, v, tokens, stream) : read_d<D, false>(c, bt, k, v, tokens, stream))
    return c.dim == 64 ? CALL(64) : (c.dim == 128 ? CALL(128) : CALL(256));
#undef CALL
}

}  // namespace dq
