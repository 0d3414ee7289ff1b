// Filling and reading the paged 4-bit key/value cache (geometry: cache4.hpp).
// A head's vector is quantized as a row of the group-wise quantizer at b = 4
// ("量化" tutorial, aiknowledge.cn, exercise 1 of its exercises): per group of g
// dimensions s = fl32(max / 7) (1.0 replaces a zero max), q = clip(rint(fl32(
// v / s)), -8, 7), code u = q + 8; a group with a NaN or an infinity gets a NaN
// scale and q = 0.
//
// Both kernels are bound by memory and by the chain of loads that finds a token's
// place (its sequence, the sequence's length, the page).  A workgroup has one kv
// head of 2048 / D consecutive tokens (a page has their codes and scales next to
// each other, so each wave writes and reads whole lines); a thread has 8 dimensions
// of the key and of the value, D/8 neighbouring threads a vector, g/8 of them a
// group, whose maximum is a butterfly over those lanes.  6207 tokens of 8 heads of
// 128 in bf16, g = 64: append (25 MB in, 7 MB out) 14.1 us, 2.3 TB/s, read (the
// reverse) 10.0 us, 3.2 TB/s; 32 tokens 4.8 and 3.5 us.  (A workgroup per two tokens, all
// heads: 15.8 and 11.6 us, for a page's lines are then written two tokens at a
// time; 32 tokens 4.1 and 3.7.)  About half of the append's time is vector work.
// The read of heads of 256 picks a word by a lane's bit, for which the compiler keeps
// the words in 16 KB of LDS; not measured against a select.
#include "cache4.hpp"
#include "common.hpp"
#include "launch_serving.hpp"
#include "quant_rule.hpp"

namespace dq {

namespace {

constexpr int kThreads = 256;

// The place of token row t: -2 for one of no sequence, -1 for one that the cache
// does not hold.  All threads of the wave take part, kParts neighbours with the same
// t, the tokens of a wave being consecutive: with up to 64 sequences each lane looks
// at the start of one, so the search is one load (the 32 tokens of a decode step,
// searched by halving: 5.4 us instead of 4.8).
template <int kParts>
__device__ __forceinline__ int64_t find_slot(const Cache4& c, const Cache4Batch& bt, int64_t t, int64_t tokens)
{
    int64_t b = 0;
    if (bt.count <= kWave) {
        const int lane = threadIdx.x % kWave;
        const int32_t start = bt.starts[lane < bt.count ? lane : bt.count - 1];
        const int64_t t0 = t - lane / kParts;
#pragma unroll
        for (int i = 0; i < kWave / kParts; ++i) {
            const int before = __popcll(__ballot(lane < bt.count && start <= t0 + i));
            if (lane / kParts == i) b = before > 0 ? before - 1 : 0;
        }
    } else {
        b = cache4_sequence(bt, t);
    }
    int64_t first, n;
    cache4_rows(bt, b, tokens, first, n);
    if (t < first || t >= first + n) return -2;
    return cache4_slot(c, bt, b, (int64_t)bt.lens[b] - n + (t - first));
}

// Where the parts of (page, head, token) begin: its code row, and the scale of its
// first group (the next group's is P floats on).
struct Place {
    int64_t row, scale;
};
template <int D>
__device__ __forceinline__ Place place_of(const Cache4& c, int64_t slot, int head, int group_shift)
{
    const int64_t block = (slot >> c.page_shift) * c.heads + head;
    const int64_t off = slot & ((1LL << c.page_shift) - 1);
    return {((block << c.page_shift) + off) * (D / 8),
            (((block * D) >> group_shift) << c.page_shift) + off};
}

// 8 elements as they lie in memory.
template <bool BF16>
struct Raw {
    uint4 d[BF16 ? 1 : 2];
    __device__ __forceinline__ void floats(float (&x)[8]) const
    {
        const uint32_t u[4] = {d[0].x, d[0].y, d[0].z, d[0].w};
        if constexpr (BF16) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[2 * e] = __uint_as_float(u[e] << 16);
                x[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
            }
        } else {
            const uint32_t w[4] = {d[1].x, d[1].y, d[1].z, d[1].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[e] = __uint_as_float(u[e]);
                x[4 + e] = __uint_as_float(w[e]);
            }
        }
    }
};
template <bool BF16>
__device__ __forceinline__ Raw<BF16> load8(const void* p, int64_t off)
{
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + off * (BF16 ? 2 : 4));
    Raw<BF16> r;
    r.d[0] = src[0];
    if constexpr (!BF16) r.d[1] = src[1];
    return r;
}

// The 8 codes of a thread (LSB first) and its group's scale.
template <bool BF16>
__device__ __forceinline__ uint32_t quantize8(const Raw<BF16>& raw, int group_threads, float* scale)
{
    float x[8], q[8];
    raw.floats(x);
    uint32_t amax = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = max(amax, __float_as_uint(x[e]) & 0x7fffffffu);
    for (int o = group_threads >> 1; o > 0; o >>= 1)
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
    *scale = s;
    clipped_quotients(x, s, __builtin_amdgcn_rcpf(s), quotient_margin(8.0f), 7.0f, q);
    // four codes at a time as the exact fp32 sum of 16^e (q + 8)
    float lo = 34952.0f, hi = 34952.0f;  // 0x8888
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        lo = fmaf(q[e], (float)(1 << (4 * e)), lo);
        hi = fmaf(q[4 + e], (float)(1 << (4 * e)), hi);
    }
    return zero ? 0x88888888u : (uint32_t)hi << 16 | (uint32_t)lo;
}

template <int D, bool BF16>
__global__ __launch_bounds__(kThreads) void cache4_append_kernel(
    Cache4 c, Cache4Batch bt, const void* __restrict__ k, const void* __restrict__ v,
    int64_t tokens, int64_t from_token, int64_t k_stride, int64_t v_stride)
{
    constexpr int kParts = D / 8;
    constexpr int kPer = D / 16;               // value codes of a c (cache4.hpp)
    constexpr int kRun = kPer < 8 ? kPer : 8;  // of them in a word
    __shared__ __attribute__((aligned(16))) uint32_t turn[kThreads];
    const int64_t t = from_token + (int64_t)blockIdx.x * (kThreads / kParts) + threadIdx.x / kParts;
    const int part = threadIdx.x % kParts;
    const int head = blockIdx.y;
    const int64_t at = (int64_t)head * D + part * 8;
    const int64_t row = t < tokens ? t : tokens - 1;
    const Raw<BF16> rk = load8<BF16>(k, row * k_stride + at), rv = load8<BF16>(v, row * v_stride + at);
    const int64_t slot = find_slot<kParts>(c, bt, t, tokens);

    const int group_shift = 31 - __builtin_clz(c.group);
    const int group_threads = c.group >> 3;
    float sk, sv;
    const uint32_t wk = quantize8<BF16>(rk, group_threads, &sk);
    const uint32_t wv = quantize8<BF16>(rv, group_threads, &sv);

    // keys: dimensions 8 part .. = 32 i + 8 r are word r (D/32) + i.
    // values: dimension 8 part + e is 16 j + c with j = part / 2, c = 8 (part & 1)
    // + e, and word w holds codes 8 w + n = c (D/16) + j: the words of a vector
    // change hands through LDS, those of one half of the c's next to each other (a
    // vector is within a wave, whose LDS accesses are in order)
    uint32_t* const mine = turn + (threadIdx.x - part);
    mine[(part & 1) * kPer + (part >> 1)] = wv;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int c0 = part * 8 / kPer;
    const uint4* from = reinterpret_cast<const uint4*>(mine + (c0 >> 3) * kPer + part * 8 % kPer);
    uint32_t x8[kRun];
#pragma unroll
    for (int e = 0; e < kRun; e += 4) {
        const uint4 d = from[e / 4];
        x8[e] = d.x, x8[e + 1] = d.y, x8[e + 2] = d.z, x8[e + 3] = d.w;
    }
    uint32_t w = 0;
#pragma unroll
    for (int n = 0; n < 8; ++n) w |= ((x8[n % kRun] >> (4 * ((c0 + n / kRun) & 7))) & 15u) << (4 * n);

    if (slot < 0) return;
    const Place p = place_of<D>(c, slot, head, group_shift);
    c.k_codes[p.row + (part & 3) * (D / 32) + (part >> 2)] = wk;
    c.v_codes[p.row + part] = w;
    if ((part & (group_threads - 1)) == 0) {
        const int64_t o = p.scale + ((int64_t)((part * 8) >> group_shift) << c.page_shift);
        c.k_scales[o] = sk;
        c.v_scales[o] = sv;
    }
}

// Elements of an output vector.
template <bool BF16>
__device__ __forceinline__ void store8(void* dst, int64_t o, const float (&x)[8])
{
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

template <int D, bool BF16>
__global__ __launch_bounds__(kThreads) void cache4_read_kernel(Cache4 c, Cache4Batch bt,
                                                               void* __restrict__ k,
                                                               void* __restrict__ v, int64_t tokens,
                                                               int64_t from_token)
{
    constexpr int kParts = D / 8;
    constexpr int kWords = D / 64 * 4;  // of the 8 c's of a thread's value dimensions
    const int64_t t = from_token + (int64_t)blockIdx.x * (kThreads / kParts) + threadIdx.x / kParts;
    const int part = threadIdx.x % kParts;
    const int head = blockIdx.y;
    const int64_t slot = find_slot<kParts>(c, bt, t, tokens);
    if (slot == -2) return;
    const int64_t o = (t * c.heads + head) * D + part * 8;
    float x[8], y[8];
    if (slot < 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = y[e] = __uint_as_float(0x7fc00000u);
    } else {
        const int group_shift = 31 - __builtin_clz(c.group);
        const Place p = place_of<D>(c, slot, head, group_shift);
        const uint32_t wk = c.k_codes[p.row + (part & 3) * (D / 32) + (part >> 2)];
        const uint4* src = reinterpret_cast<const uint4*>(c.v_codes + p.row + (part & 1) * kWords);
        uint32_t w[kWords];
#pragma unroll
        for (int e = 0; e < kWords; e += 4) {
            const uint4 d = src[e / 4];
            w[e] = d.x, w[e + 1] = d.y, w[e + 2] = d.z, w[e + 3] = d.w;
        }
        const int64_t so = p.scale + ((int64_t)((part * 8) >> group_shift) << c.page_shift);
        const float sk = c.k_scales[so], sv = c.v_scales[so];
        const int j = part >> 1;  // the code of each c
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            uint32_t u;
            if constexpr (D == 64)
                u = w[e / 2] >> (16 * (e & 1) + 4 * j);
            else if constexpr (D == 128)
                u = w[e] >> (4 * j);
            else
                u = (j & 8 ? w[2 * e + 1] : w[2 * e]) >> (4 * (j & 7));
            x[e] = (float)((int32_t)((wk >> (4 * e)) & 15u) - 8) * sk;
            y[e] = (float)((int32_t)(u & 15u) - 8) * sv;
        }
    }
    store8<BF16>(k, o, x);
    store8<BF16>(v, o, y);
}

// Launches for the tokens from, from + kLaunchTokens, ... (a launch has at most
// 2^32 - 1 threads a dimension).
constexpr int64_t kLaunchTokens = 1LL << 26;
template <class F>
hipError_t by_tokens(const Cache4& c, int64_t tokens, F launch)
{
    for (int64_t from = 0; from < tokens; from += kLaunchTokens) {
        const int64_t n = tokens - from < kLaunchTokens ? tokens - from : kLaunchTokens;
        launch(dim3((unsigned)ceil_div(n, kThreads / (c.dim / 8)), (unsigned)c.heads), from);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_cache4_append(const Cache4& c, const Cache4Batch& bt, const void* k,
                                const void* v, bool bf16, int64_t tokens, int64_t k_stride,
                                int64_t v_stride, hipStream_t stream)
{
#define CALL(D) \
    (bf16 ? cache4_append_kernel<D, true> : cache4_append_kernel<D, false>)
    const auto kernel = c.dim == 64 ? CALL(64) : (c.dim == 128 ? CALL(128) : CALL(256));
    return by_tokens(c, tokens, [&](dim3 grid, int64_t from) {
        kernel<<<grid, kThreads, 0, stream>>>(c, bt, k, v, tokens, from, k_stride, v_stride);
    });
#undef CALL
}

hipError_t launch_cache4_read(const Cache4& c, const Cache4Batch& bt, void* k, void* v, bool bf16,
                              int64_t tokens, hipStream_t stream)
{
#define CALL(D) \
    (bf16 ? cache4_read_kernel<D, true> : cache4_read_kernel<D, false>)
    const auto kernel = c.dim == 64 ? CALL(64) : (c.dim == 128 ? CALL(128) : CALL(256));
    return by_tokens(c, tokens, [&](dim3 grid, int64_t from) {
        kernel<<<grid, kThreads, 0, stream>>>(c, bt, k, v, tokens, from);
    });
#undef CALL
}

}  // namespace dq
