// Causal attention of new queries over the paged 4-bit cache (cache4.hpp):
//   o[i,h] = sum_t p_t vhat[t] / sum_t p_t,  p_t = exp(scale q[i,h] . khat[t] - max),
// over the cached positions t up to query i's own, khat / vhat = q4 * group scale.
//
// One wave takes 16 rows (query, head of one kv head's group) and walks the
// positions 32 at a time with the running maximum and sum of a softmax.  Both
// products run on v_mfma_f32_16x16x32_f16 in transposed form, S^T = K Q^T and
// O^T = V^T P^T, so that a lane holds one row (lane & 15) throughout: the
// softmax is in-lane but for two steps across the four lanes of a row, and S^T
// comes out in the lane and order in which P^T goes in.
//   * The codes are exact in fp16 (u | 0x6400 is 1024 + u; the offset comes off
//     exactly).  Each row of q is multiplied by a power of two that puts its
//     largest element in [2^14, 2^15): exact for every element above 2^-28 of
//     it.  A group's partial dot products are scaled in fp32.
//   * p * (value scale) is rounded once, to fp16, after multiplication by a
//     power of two that puts the largest value scale seen so far in [2^14,
//     2^15): relative error 2^-11 down to 2^-29 of the largest.
#include "cache4.hpp"
#include "common.hpp"
#include "launch_serving.hpp"

namespace dq {

namespace {

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ uint32_t u32_of(f16x2_t v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ f16x2_t f16x2_of(uint32_t v) { return __builtin_bit_cast(f16x2_t, v); }

// The codes in bits 0..3 and 16..19 of v as fp16 (u - 8), exact.
__device__ __forceinline__ uint32_t low_codes(uint32_t v)
{
    const f16x2_t h = f16x2_of((v & 0x000f000fu) | 0x64006400u);  // 1024 + u
    return u32_of(h - (f16x2_t){(_Float16)1032.0f, (_Float16)1032.0f});
}
// The codes in bits 4..7 and 20..23.
__device__ __forceinline__ uint32_t high_codes(uint32_t v)
{
    const f16x2_t h = f16x2_of((v & 0x00f000f0u) | 0x64006400u);  // 1024 + 16 u
    const _Float16 s = (_Float16)0.0625f, o = (_Float16)-72.0f;
    return u32_of(__builtin_elementwise_fma(h, (f16x2_t){s, s}, (f16x2_t){o, o}));
}

// The 8 codes of a word as an fp16 operand, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ f16x8_t word_codes(uint32_t w)
{
    const uint32_t x = w >> 8;
    return __builtin_bit_cast(f16x8_t, (u32x4_t){low_codes(w), high_codes(w), low_codes(x), high_codes(x)});
}

// max over the four lanes l, l ^ 16, l ^ 32, l ^ 48
__device__ __forceinline__ float row_max(float v)
{
    v = fmaxf(v, __shfl_xor(v, 16, kWave));
    return fmaxf(v, __shfl_xor(v, 32, kWave));
}
__device__ __forceinline__ float row_sum(float v)
{
    v += __shfl_xor(v, 16, kWave);
    return v + __shfl_xor(v, 32, kWave);
}

// 2^n for n clamped to fp32's normal range
__device__ __forceinline__ float pow2(int n)
{
    n = n < -126 ? -126 : (n > 127 ? 127 : n);
    return __uint_as_float((uint32_t)(n + 127) << 23);
}
// floor(log2 v) of a normal v (-127 for zero and subnormals, 128 for inf / NaN)
__device__ __forceinline__ int exponent(float v)
{
    return (int)((__float_as_uint(v) >> 23) & 0xff) - 127;
}

struct AttnArgs {
    Cache4 c;
    Cache4Batch bt;
    const uint16_t* q;
    int64_t q_stride;
    uint16_t* out;
    int64_t tokens;
    int32_t q_heads;
    float scale_log2;
};

template <int D, int G>
__global__ __launch_bounds__(kWave) void cache4_attention_kernel(AttnArgs a)
{
    constexpr int NC = D / 32;  // 32-dimension steps of a dot product
    constexpr int NG = D / G;   // groups of a head
    constexpr int GC = G / 32;  // steps of a group
    constexpr int NT = D / 16;  // 16-dimension tiles of the output
    constexpr int VW = D / 128 > 0 ? D / 128 : 1;  // value words a lane reads of a token
    const int lane = threadIdx.x;
    const int r16 = lane & 15;
    const int kg = lane >> 4;
    const int64_t b = blockIdx.z;
    const int kvh = blockIdx.y;
    const int per = a.q_heads / a.c.heads;  // query heads of a kv head
    const int shift = a.c.page_shift;
    const int64_t P = 1LL << shift;

    int64_t first, nq;
    cache4_rows(a.bt, b, a.tokens, first, nq);
    const int64_t rows = nq * per;
    int64_t len = a.bt.lens[b];
    const bool bad_len = len > a.bt.width << shift;
    if (len < 0 || bad_len) len = 0;

    for (int64_t r0 = (int64_t)blockIdx.x * 16; r0 < rows; r0 += (int64_t)gridDim.x * 16) {
        const int64_t row = r0 + r16;
        const bool live = row < rows;
        const int64_t qi = live ? row / per : 0;
        const int head = kvh * per + (live ? (int)(row % per) : 0);
        const int64_t limit = live ? len - nq + qi : -1;  // last position the row sees
        const int64_t last_row = r0 + 15 < rows ? r0 + 15 : rows - 1;
        const int64_t end = len - nq + last_row / per + 1;

        // q row -> fp16 operands, scaled by a power of two
        const uint16_t* qp = a.q + (first + qi) * a.q_stride + (int64_t)head * D + 8 * kg;
        uint4 qr[NC];
        float qmax = 0.0f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            qr[i] = *reinterpret_cast<const uint4*>(qp + 32 * i);
            const uint32_t u[4] = {qr[i].x, qr[i].y, qr[i].z, qr[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // as integers: a NaN is larger than everything and stays visible
                const uint32_t lo = (u[e] << 16) & 0x7fffffffu, hi = u[e] & 0x7fff0000u;
                qmax = __uint_as_float(max(__float_as_uint(qmax), max(lo, hi)));
            }
        }
        {
            uint32_t m = __float_as_uint(qmax);
            m = max(m, (uint32_t)__shfl_xor((int)m, 16, kWave));
            m = max(m, (uint32_t)__shfl_xor((int)m, 32, kWave));
            qmax = __uint_as_float(m);
        }
        const int ue = min(14 - exponent(qmax), 126);
        const float up = pow2(ue);
        const float logit = a.scale_log2 * pow2(-ue);
        f16x8_t qf[NC];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const uint32_t u[4] = {qr[i].x, qr[i].y, qr[i].z, qr[i].w};
            float f[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f[2 * e] = __uint_as_float(u[e] << 16) * up;
                f[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u) * up;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {  // the order of word_codes
                qf[i][2 * e] = (_Float16)f[e];
                qf[i][2 * e + 1] = (_Float16)f[e + 4];
            }
        }

        float m = -INFINITY, l = 0.0f;
        int ve = -112;  // exponent that the value scales are measured against
        f32x4_t o[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) o[j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};

        for (int64_t t0 = 0; t0 < end; t0 += 32) {
            float s[8];
            float vs[8][NG];
            uint32_t vw[8][VW];
            float vtop = 0.0f;
#pragma unroll
            for (int tile = 0; tile < 2; ++tile) {
                // 16 positions of one page; past the end, the last one again
                const int64_t tt = t0 + 16 * tile < end ? t0 + 16 * tile : (end - 1) & ~15LL;
                int64_t page = a.bt.table[b * a.bt.width + (tt >> shift)];
                const bool bad = page < 0 || page >= a.c.pages;
                if (bad) page = 0;
                const int64_t off = tt & (P - 1);
                const int64_t block = page * a.c.heads + kvh;
                const int64_t crow = ((block << shift) + off) * (D / 8);
                const uint32_t* kp = a.c.k_codes + crow + r16 * (D / 8) + kg * NC;
                uint32_t kw[NC];
#pragma unroll
                for (int i = 0; i < NC; ++i) kw[i] = kp[i];
                const float* ksc = a.c.k_scales + ((block * NG) << shift) + off + 4 * kg;
                const float* vsc = a.c.v_scales + ((block * NG) << shift) + off + 4 * kg;
                f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    f32x4_t part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < GC; ++i)
                        part = __builtin_amdgcn_mfma_f32_16x16x32_f16(word_codes(kw[g * GC + i]),
                                                                      qf[g * GC + i], part, 0, 0, 0);
                    const float4 ks = *reinterpret_cast<const float4*>(ksc + ((int64_t)g << shift));
                    const float4 v4 = *reinterpret_cast<const float4*>(vsc + ((int64_t)g << shift));
                    acc[0] = fmaf(ks.x, part[0], acc[0]);
                    acc[1] = fmaf(ks.y, part[1], acc[1]);
                    acc[2] = fmaf(ks.z, part[2], acc[2]);
                    acc[3] = fmaf(ks.w, part[3], acc[3]);
                    vs[4 * tile][g] = v4.x, vs[4 * tile + 1][g] = v4.y;
                    vs[4 * tile + 2][g] = v4.z, vs[4 * tile + 3][g] = v4.w;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int64_t pos = t0 + 16 * tile + 4 * kg + e;
                    float x = acc[e] * logit;
                    if (bad) x = __uint_as_float(0x7fc00000u);
                    s[4 * tile + e] = pos <= limit ? x : -INFINITY;
                    if (pos < end) {
#pragma unroll
                        for (int g = 0; g < NG; ++g) vtop = fmaxf(vtop, vs[4 * tile + e][g]);
                    }
                    const uint32_t* vp = a.c.v_codes + crow + (4 * kg + e) * (D / 8);
                    if constexpr (D == 64) {
                        vw[4 * tile + e][0] = reinterpret_cast<const uint16_t*>(vp)[r16];
                    } else {
#pragma unroll
                        for (int i = 0; i < VW; ++i) vw[4 * tile + e][i] = vp[r16 * VW + i];
                    }
                }
            }
            // value scales' common power of two
            vtop = row_max(vtop);
            const int vn = exponent(vtop) > ve ? exponent(vtop) : ve;
            const float vfac = pow2(14 - vn);
            // running maximum and sum
            float mx = s[0];
#pragma unroll
            for (int e = 1; e < 8; ++e) mx = fmaxf(mx, s[e]);
            const float mn = fmaxf(m, row_max(mx));
            const float base = mn == -INFINITY ? 0.0f : mn;
            const float alpha = __builtin_amdgcn_exp2f(m - base);
            const float oscale = alpha * pow2(ve - vn);
            m = mn;
            ve = vn;
            float p[8];
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                p[e] = __builtin_amdgcn_exp2f(s[e] - base);
                sum += p[e];
            }
            l = fmaf(l, alpha, sum);
#pragma unroll
            for (int j = 0; j < NT; ++j) o[j] *= oscale;
            f16x8_t pf[NG];
#pragma unroll
            for (int g = 0; g < NG; ++g) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int64_t pos = t0 + 16 * (e >> 2) + 4 * kg + (e & 3);
                    pf[g][e] = (_Float16)(pos <= limit ? p[e] * (vs[e][g] * vfac) : 0.0f);
                }
            }
            // tile j: nibble j of the lane's codes of 8 positions, pairs of positions
#pragma unroll
            for (int i = 0; i < VW; ++i) {
#pragma unroll
                for (int n = 0; n < (D == 64 ? 2 : 4); ++n) {
                    const uint32_t sel = 0x0c000c00u | ((uint32_t)(4 + n) << 16) | (uint32_t)n;
                    uint32_t lo[4], hi[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t v = __builtin_amdgcn_perm(vw[2 * e + 1][i], vw[2 * e][i], sel);
                        lo[e] = low_codes(v);
                        hi[e] = high_codes(v);
                    }
                    const int j = 8 * i + 2 * n;
                    const f16x8_t vl = __builtin_bit_cast(f16x8_t, (u32x4_t){lo[0], lo[1], lo[2], lo[3]});
                    const f16x8_t vh = __builtin_bit_cast(f16x8_t, (u32x4_t){hi[0], hi[1], hi[2], hi[3]});
                    o[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vl, pf[16 * j / G], o[j], 0, 0, 0);
                    o[j + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vh, pf[16 * (j + 1) / G], o[j + 1], 0, 0, 0);
                }
            }
        }
        l = row_sum(l);
        float inv = l > 0.0f ? pow2(ve - 14) / l : (l == 0.0f ? 0.0f : l);  // NaN stays
        if (bad_len) inv = __uint_as_float(0x7fc00000u);
        if (live) {
            uint16_t* op = a.out + ((first + qi) * a.q_heads + head) * D + 4 * kg;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                uint32_t w[2];
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    w[e] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)(o[j][2 * e] * inv)) |
                           ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)(o[j][2 * e + 1] * inv)) << 16);
                *reinterpret_cast<uint2*>(op + 16 * j) = make_uint2(w[0], w[1]);
            }
        }
    }
}

template <int D, int G>
hipError_t launch_dg(const AttnArgs& a, int64_t max_q, hipStream_t stream)
{
    const int64_t tiles = ceil_div(max_q * (a.q_heads / a.c.heads), 16);
    const dim3 grid((unsigned)(tiles < 65535 ? tiles : 65535), (unsigned)a.c.heads,
                    (unsigned)a.bt.count);
    cache4_attention_kernel<D, G><<<grid, kWave, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

size_t cache4_attention_workspace(const Cache4& c, int64_t count, int64_t tokens,
                                  int q_heads, int64_t max_q, int64_t max_len)
{
    (void)c, (void)count, (void)tokens, (void)q_heads, (void)max_q, (void)max_len;
    return 0;
}

hipError_t launch_cache4_attention(const Cache4& c, const Cache4Batch& bt, const uint16_t* q,
                                   int64_t tokens, int64_t q_stride, int q_heads, float scale,
                                   int64_t max_q, int64_t max_len, uint16_t* out, void* workspace,
                                   hipStream_t stream)
{
    (void)max_len;
    (void)workspace;
    const AttnArgs a{c, bt, q, q_stride, out, tokens, q_heads, scale * kLog2e};
    switch (c.dim * 1000 + c.group) {
    case 64032: return launch_dg<64, 32>(a, max_q, stream);
    case 64064: return launch_dg<64, 64>(a, max_q, stream);
    case 128032: return launch_dg<128, 32>(a, max_q, stream);
    case 128064: return launch_dg<128, 64>(a, max_q, stream);
    case 128128: return launch_dg<128, 128>(a, max_q, stream);
    case 256032: return launch_dg<256, 32>(a, max_q, stream);
    case 256064: return launch_dg<256, 64>(a, max_q, stream);
    case 256128: return launch_dg<256, 128>(a, max_q, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace dq
