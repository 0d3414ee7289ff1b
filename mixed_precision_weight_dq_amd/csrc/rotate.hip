// Rotary positions applied to tokens [tokens, heads, D] (rope.hpp).  Angles in
// fp64, their sine and cosine and the products in fp32, one rounding to the
// tokens' type.
//
// Bound by memory.  rotate_kernel: a thread has 8 pairs of a token (two pieces of 8 elements)
// and walks some of its heads, so that 8 sines and cosines serve all of them; pieces of
// neighbouring threads are neighbours in memory.  6000 tokens of 40 heads of 128 in bf16
// (123 MB in and out) 26.8 us, 4.6 TB/s; half of each head, interleaved 30.4 us; 3000 in fp32 36 us.
//
// rotate_any_kernel has one pair at a time: for the sizes, strides and addresses that pieces
// do not fit (there it takes 51 and 59 us for the first two), and for small calls, where eight
// sines one after another are the longest wait: 1 x 32 heads of 128 2.5 us (pieces 3.0).
#include "common.hpp"
#include "launch_serving.hpp"

namespace dq {

namespace {

constexpr int kThreads = 256;
constexpr int64_t kLaunchThreads = 1LL << 31;  // (a launch has at most 2^32 - 1)

struct RotateArgs {
    Rope rope;
    const void* x;
    void* out;
    const int32_t* positions;
    int64_t x_token, x_head, out_token, out_head;  // strides in elements
    int64_t from;      // first token of the launch
    uint32_t tokens;   // of the launch
    uint32_t slots;    // threads of a token's head
    uint32_t lanes;    // heads of a token that are worked on side by side
    int32_t heads, dim;
};

// Thread g of the launch: slot, then lane, then token.
__device__ __forceinline__ bool rotate_place(const RotateArgs& a, uint32_t& slot, uint32_t& lane, int64_t& token)
{
    const uint32_t g = blockIdx.x * kThreads + threadIdx.x;
    const uint32_t unit = g / a.slots;
    slot = g - unit * a.slots;
    const uint32_t t = unit / a.lanes;
    lane = unit - t * a.lanes;
    token = a.from + t;
    return t < a.tokens;
}

__device__ __forceinline__ void rotate_turn(const Rope& r, int32_t pos, int i, float& c, float& s)
{
    sincospif(2.0f * (float)turn_fraction(pos, r.turns[i]), &s, &c);
    c *= (float)r.factor;
    s *= (float)r.factor;
}

// A piece of 8 elements.
template <bool BF16>
struct Piece {
    uint4 d[BF16 ? 1 : 2];
    __device__ __forceinline__ void load(const void* p, int64_t off)
    {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + off * (BF16 ? 2 : 4));
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i) d[i] = src[i];
    }
    __device__ __forceinline__ void store(void* p, int64_t off) const
    {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<char*>(p) + off * (BF16 ? 2 : 4));
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i) dst[i] = d[i];
    }
    __device__ __forceinline__ void floats(float (&x)[8]) const
    {
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i) {
            const uint32_t u[4] = {d[i].x, d[i].y, d[i].z, d[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (BF16) {
                    x[2 * e] = __uint_as_float(u[e] << 16);
                    x[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
                } else {
                    x[4 * i + e] = __uint_as_float(u[e]);
                }
            }
        }
    }
    __device__ __forceinline__ void set(const float (&x)[8])
    {
        uint32_t u[BF16 ? 4 : 8];
#pragma unroll
        for (int e = 0; e < (BF16 ? 4 : 8); ++e) {
            if constexpr (BF16)
                u[e] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * e]) |
                       (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * e + 1]) << 16;
            else
                u[e] = __float_as_uint(x[e]);
        }
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i) d[i] = make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
    }
};

template <bool BF16, bool kInter, int kDeep>  // kDeep: heads whose pieces are in flight
__global__ __launch_bounds__(kThreads) void rotate_kernel(RotateArgs a)
{
    uint32_t slot, lane;
    int64_t token;
    if (!rotate_place(a, slot, lane, token)) return;
    const int groups = a.rope.dims / 16;
    const bool turned = (int)slot < groups;
    // the slot's pieces: rotated, or the ones behind them, two by two
    const int d0 = turned ? (kInter ? 16 : 8) * (int)slot : a.rope.dims + 16 * ((int)slot - groups);
    const int d1 = turned && !kInter ? d0 + a.rope.dims / 2 : d0 + 8;
    const bool second = d1 < a.dim;
    const int64_t from = token * a.x_token, to = token * a.out_token;
    Piece<BF16> p0[kDeep], p1[kDeep];
    const auto load = [&](int h) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            const int64_t n = h + k * (int)a.lanes < a.heads ? h + k * (int)a.lanes : h;  // (the first again)
            p0[k].load(a.x, from + n * a.x_head + d0);
            p1[k].load(a.x, from + n * a.x_head + (second ? d1 : d0));
        }
    };
    load(lane);
    float c[8], s[8];
    if (turned) {
        const int32_t pos = a.positions[token];
#pragma unroll
        for (int i = 0; i < 8; ++i) rotate_turn(a.rope, pos, 8 * (int)slot + i, c[i], s[i]);
    }
    for (int h = lane; h < a.heads; h += kDeep * a.lanes) {
        if (h != (int)lane) load(h);
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            const int64_t n = h + k * (int)a.lanes;
            if (n >= a.heads) break;
            if (turned) {
                float x[8], y[8];
                p0[k].floats(x);
                p1[k].floats(y);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    // pair i: an element of each piece, or two neighbours
                    float& u = !kInter ? x[i] : (i < 4 ? x[2 * (i & 3)] : y[2 * (i & 3)]);
                    float& v = !kInter ? y[i] : (i < 4 ? x[2 * (i & 3) + 1] : y[2 * (i & 3) + 1]);
                    const float p = u, q = v;
                    u = fmaf(p, c[i], -q * s[i]);
                    v = fmaf(q, c[i], p * s[i]);
                }
                p0[k].set(x);
                p1[k].set(y);
            }
            p0[k].store(a.out, to + n * a.out_head + d0);
            if (second) p1[k].store(a.out, to + n * a.out_head + d1);
        }
    }
}

template <bool BF16>
__device__ __forceinline__ float element(const void* p, int64_t i)
{
    return BF16 ? bf16_bits_to_float(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}
template <bool BF16>
__device__ __forceinline__ void put(void* p, int64_t i, float v)
{
    if (BF16)
        static_cast<uint16_t*>(p)[i] = __builtin_bit_cast(uint16_t, (__bf16)v);
    else
        static_cast<float*>(p)[i] = v;
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void rotate_any_kernel(RotateArgs a)
{
    uint32_t slot, lane;
    int64_t token;
    if (!rotate_place(a, slot, lane, token)) return;
    const int pairs = a.rope.dims / 2;
    const bool turned = (int)slot < pairs;
    const int d0 = turned ? (a.rope.interleaved ? 2 * (int)slot : (int)slot) : pairs + (int)slot;
    const int d1 = a.rope.interleaved ? d0 + 1 : d0 + pairs;
    float c = 1.0f, s = 0.0f;
    if (turned) rotate_turn(a.rope, a.positions[token], slot, c, s);
    for (int h = lane; h < a.heads; h += a.lanes) {
        const int64_t from = token * a.x_token + h * a.x_head;
        const int64_t to = token * a.out_token + h * a.out_head;
        const float p = element<BF16>(a.x, from + d0);
        if (turned) {
            const float q = element<BF16>(a.x, from + d1);
            put<BF16>(a.out, to + d0, fmaf(p, c, -q * s));
            put<BF16>(a.out, to + d1, fmaf(q, c, p * s));
        } else {
            put<BF16>(a.out, to + d0, p);
        }
    }
}

template <int kDeep>
auto pieces_kernel(bool bf16, bool interleaved) -> void (*)(RotateArgs)
{
    return interleaved ? (bf16 ? rotate_kernel<true, true, kDeep> : rotate_kernel<false, true, kDeep>)
                       : (bf16 ? rotate_kernel<true, false, kDeep> : rotate_kernel<false, false, kDeep>);
}

}  // namespace

hipError_t launch_rotate(const Rope& rope, const void* x, bool bf16, int64_t tokens, int heads, int dim,
                         int64_t x_token, int64_t x_head, const int32_t* positions, void* out,
                         int64_t out_token, int64_t out_head, hipStream_t stream)
{
    RotateArgs a{rope, x, out, positions, x_token, x_head, out_token, out_head, 0, 0, 0, 0, heads, dim};
    const bool same = x == out && x_token == out_token && x_head == out_head;
    const int rest = same ? 0 : dim - rope.dims;  // copied
    const int64_t unit = bf16 ? 8 : 4;            // elements of 16 bytes
    // pieces, pairs: 64 x 32 heads of 128 3.2 us, 2.8; 160 x 32 (328 k threads of pairs) 3.4, 3.3; 200 x 32
    // (410 k) 3.4, 3.7; 500 x 32 4.2, 4.8; half of a head, 64 x 40 (246 k) 3.2, 3.0, 128 x 40 (492 k) 3.4, 3.8
    constexpr int64_t kFewThreads = 3 << 17;
    const bool pieces = tokens * heads * (int64_t)(rope.dims / 2 + rest) > kFewThreads &&
                        rope.dims % 16 == 0 && dim % 8 == 0 && x_token % unit == 0 && x_head % unit == 0 &&
                        out_token % unit == 0 && out_head % unit == 0 &&
                        ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(out)) & 15) == 0;
    a.slots = pieces ? rope.dims / 16 + ceil_div(rest, 16) : rope.dims / 2 + rest;
    // Heads of a thread: as many as leave kFill threads (6000 x 40 heads of 128 26.8 us; 2^16 threads 26.5,
    // 2^20 37.2; 1700 x 36 of 256 13.1; 14.2, 18.4), four of them in flight (one 28.0 us, two 28.9,
    // eight 26.8 and 40 in fp32 for 36); a thread with one head asks for no more.
    constexpr int64_t kFill = 1 << 18;
    const int64_t most = tokens * heads * (int64_t)a.slots / kFill;
    const int per = (int)(most < 1 ? 1 : (most > 8 ? 8 : most));
    a.lanes = ceil_div(heads, per);
    const int64_t token_threads = (int64_t)a.slots * a.lanes;
    const int64_t step = kLaunchThreads / token_threads;
    for (int64_t from = 0; from < tokens; from += step) {
        a.from = from;
        a.tokens = (uint32_t)(tokens - from < step ? tokens - from : step);
        const dim3 grid((unsigned)ceil_div(a.tokens * token_threads, kThreads));
        if (pieces)
            (per == 1 ? pieces_kernel<1>(bf16, rope.interleaved) : pieces_kernel<4>(bf16, rope.interleaved))
                <<<grid, kThreads, 0, stream>>>(a);
        else
            (bf16 ? rotate_any_kernel<true> : rotate_any_kernel<false>)<<<grid, kThreads, 0, stream>>>(a);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace dq
