// Attention of drafted tokens over the paged 4-bit cache: every token sees the cached
// context, and of the call's own tokens those whose bits its mask has.
//
// One wave per token and query head; a lane has the dot product of one of 64
// positions, then the wave's lanes the dimensions of the output.
#include "cache4.hpp"
#include "common.hpp"
#include "launch_serving.hpp"

namespace dq {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kMaxLen = 0x7fff0000;

struct TreeArgs {
    Cache4 c;
    Cache4Batch bt;
    const uint16_t* q;
    int64_t q_stride;
    uint16_t* out;
    int64_t tokens;
    int32_t q_heads;
    float scale_log2;
    const int32_t* mask;
    int64_t words;
};

template <int D>
__global__ __launch_bounds__(kWave) void cache4_tree_kernel(TreeArgs a)
{
    __shared__ float qs[D];
    __shared__ float ps[kWave];
    __shared__ int64_t at[kWave];
    const int lane = threadIdx.x;
    const int head = blockIdx.y, kvh = head / (a.q_heads / a.c.heads);
    const int gshift = 31 - __builtin_clz(a.c.group);
    const int64_t P = 1LL << a.c.page_shift;
    for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
        const int64_t b = cache4_sequence(a.bt, t);
        int64_t first, n;
        cache4_rows(a.bt, b, a.tokens, first, n);
        if (t < first || t >= first + n) continue;
        int64_t len = a.bt.lens[b];
        const bool bad = len > kMaxLen || len > a.bt.width * P;
        if (len < 0 || bad) len = 0;
        const int64_t context = len - n;
        __syncthreads();
        for (int d = lane; d < D; d += kWave)
            qs[d] = bf16_bits_to_float(a.q[t * a.q_stride + (int64_t)head * D + d]) * a.scale_log2;
        __syncthreads();
        float m = -INFINITY, l = 0.0f, o[D / kWave];
#pragma unroll
        for (int i = 0; i < D / kWave; ++i) o[i] = 0.0f;
        for (int64_t t0 = 0; t0 < len; t0 += kWave) {
            const int64_t pos = t0 + lane, j = pos - context;
            bool sees = pos < len;
            if (sees && j >= 0) sees = (j >> 5) < a.words && (a.mask[t * a.words + (j >> 5)] >> (j & 31) & 1);
            float s = -INFINITY;
            int64_t slot = -1;
            if (sees) {
                slot = cache4_slot(a.c, a.bt, b, pos);
                s = __uint_as_float(0x7fc00000u);
                if (slot >= 0) {
                    const int64_t block = (slot >> a.c.page_shift) * a.c.heads + kvh, off = slot & (P - 1);
                    const uint32_t* k = a.c.k_codes + (block * P + off) * (D / 8);
                    s = 0.0f;
                    for (int w = 0; w < D / 8; ++w) {
                        const int d0 = (w % (D / 32)) * 32 + w / (D / 32) * 8;
                        const float sc = a.c.k_scales[((block * D >> gshift) + (d0 >> gshift)) * P + off];
                        float dot = 0.0f;
                        for (int e = 0; e < 8; ++e) dot += ((int)(k[w] >> (4 * e) & 15) - 8) * qs[d0 + e];
                        s += dot * sc;
                    }
                }
            }
            float mx = s;
            for (int x = kWave / 2; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor(mx, x, kWave));
            const float mn = fmaxf(m, mx), base = mn == -INFINITY ? 0.0f : mn;
            const float p = exp2f(s - base), alpha = exp2f(m - base);
            float sum = p;
            for (int x = kWave / 2; x > 0; x >>= 1) sum += __shfl_xor(sum, x, kWave);
            l = l * alpha + sum;
            m = mn;
            ps[lane] = p;
            at[lane] = sees ? slot : -2;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < D / kWave; ++i) {
                const int d = i * kWave + lane, place = (d % 16) * (D / 16) + d / 16;
                o[i] *= alpha;
                for (int e = 0; e < kWave; ++e) {
                    if (at[e] < 0) continue;
                    const int64_t block = (at[e] >> a.c.page_shift) * a.c.heads + kvh, off = at[e] & (P - 1);
                    const uint32_t w = a.c.v_codes[(block * P + off) * (D / 8) + place / 8];
                    const float sc = a.c.v_scales[((block * D >> gshift) + (d >> gshift)) * P + off];
                    o[i] += ps[e] * (((int)(w >> (4 * (place % 8)) & 15) - 8) * sc);
                }
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < D / kWave; ++i) {
            const float v = bad ? __uint_as_float(0x7fc00000u) : (l == 0.0f ? 0.0f : o[i] / l);
            a.out[(t * a.q_heads + head) * D + i * kWave + lane] = __builtin_bit_cast(uint16_t, (__bf16)v);
        }
    }
}

}  // namespace

size_t cache4_tree_workspace(const Cache4&, int64_t, int64_t, int, int64_t, int64_t) { return 0; }

hipError_t launch_cache4_tree(const Cache4& c, const Cache4Batch& bt, const uint16_t* q, int64_t tokens,
                              int64_t q_stride, int q_heads, const int32_t* mask, int64_t words,
                              float scale, int64_t, int64_t, uint16_t* out, void*, hipStream_t stream)
{
    const TreeArgs a{c, bt, q, q_stride, out, tokens, q_heads, scale * kLog2e, mask, words};
    const dim3 grid((unsigned)(tokens < 65536 ? tokens : 65536), (unsigned)q_heads);
    (c.dim == 64 ? cache4_tree_kernel<64> : (c.dim == 128 ? cache4_tree_kernel<128> : cache4_tree_kernel<256>))
        <<<grid, kWave, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace dq
